// Rotary positions, alone and on the way into a paged KV cache.
//
// Mathematics: pair i of a token's head, (a, b), becomes
//   mscale * (a cos t - b sin t, b cos t + a sin t),  t = +-pos[axis(i)] * freqs[i].
// The product is formed in float64 and reduced to half turns in (-1, 1] there
// (a float32 angle of position 10^6 is off by 0.03 rad); cos and sin of the
// remainder and the rotation are float32, rounded once to the output type.
//
// What bounds it: bytes, each element read once and written once. A thread owns
// a few pairs of one token, forms their cos and sin once and keeps them in
// registers while it walks over heads (queries, keys; values are copied on the
// way), so that the float64 work is shared by the heads and nothing but the
// tensors is read. Heads are split over gridDim.y only as far as it takes to
// fill the GPU, because every part forms its angles again.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "velox_internal.cuh"

namespace velox {

namespace {

constexpr int RT = 128;  // threads per CTA

__device__ __forceinline__ void turn(double freq, int pos, float mscale, float sign, float& c,
                                     float& s) {
    // h = t / pi as an unevaluated sum: 1/pi in two doubles, so that the
    // reduction adds nothing to the rounding of t itself
    const double inv_pi = 0.31830988618379067154, inv_pi_lo = -1.9678676675182486e-17;
    const double t = static_cast<double>(pos) * freq;
    const double h = t * inv_pi;
    const double lo = fma(t, inv_pi, -h) + t * inv_pi_lo;
    const double n = 2.0 * rint(0.5 * h);
    float sn, cs;
    sincospif(static_cast<float>((h - n) + lo), &sn, &cs);
    c = cs * mscale;
    s = sn * mscale * sign;
}

__device__ __forceinline__ int axis_pos(const RopeArgs& a, const int32_t* p, int pair) {
    const int ax = pair < a.sec0 ? 0 : (pair < a.sec01 ? 1 : 2);
    return p[ax * a.pos_axis];
}

template <bool B>
struct Const {
    __device__ constexpr operator bool() const { return B; }
};

// 8 consecutive elements
template <typename T>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16> {
    uint4 r;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        r = *reinterpret_cast<const uint4*>(p);
    }
    __device__ __forceinline__ void get(float* f) const {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
template <>
struct Chunk<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void get(float* f) const {
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
        f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
};

__device__ __forceinline__ uint32_t bf2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void put(__nv_bfloat16* p, const float* f) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(bf2(f[0], f[1]), bf2(f[2], f[3]), bf2(f[4], f[5]), bf2(f[6], f[7]));
}
__device__ __forceinline__ void put(float* p, const float* f) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ void put1(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void put1(float* p, float x) { *p = x; }

// A group's rows of one token: where row h starts, and whether it is written.
template <typename TI, typename TO>
struct Rows {
    const TI* x;
    TO* y;
    long long xh, yh;
    bool live;
    __device__ __forceinline__ Rows(const RopeArgs& a, const RopeGroup& g, int b, int n,
                                    long long slot) {
        x = static_cast<const TI*>(g.x) + b * g.xb + n * g.xn;
        xh = g.xh;
        live = true;
        if (g.to_pages) {
            live = slot >= 0;
            const long long page_id = slot >> a.page_shift, row = slot & (a.page - 1);
            y = static_cast<TO*>(g.y) +
                ((page_id * g.heads << a.page_shift) + row) * static_cast<long long>(a.d);
            yh = static_cast<long long>(a.page) * a.d;
        } else {
            y = static_cast<TO*>(g.y) + b * g.yb + n * g.yn;
            yh = g.yh;
        }
    }
};

// Rows [h0, h1) of the launch, counted over the groups, cut to group `g`.
__device__ __forceinline__ void cut(const RopeArgs& a, int g, int h0, int h1, int& lo, int& hi) {
    int first = 0;
    for (int i = 0; i < g; ++i) first += a.g[i].heads;
    lo = max(h0 - first, 0);
    hi = min(h1 - first, a.g[g].heads);
}

__device__ __forceinline__ long long token_slot(const RopeArgs& a, long long t, bool report) {
    if (!a.slots) return 0;
    const long long s = a.slots[t];
    if (s >= a.n_slots) {
        if (report && a.status) atomicOr(a.status, VELOX_STATUS_BAD_INDEX);
        return -1;
    }
    return s;
}

// 16-byte accesses. A row (a head of a token) is cut in items of two chunks (half
// layout: chunks i and i + rot/16 of the rotated part, then neighbours of the rest) or
// one (interleaved); 1 << lanes_log2 threads share a token, an item each, and keep the
// factors of their item through all heads. What is not rotated takes the same way
// past the arithmetic, so that a warp does not part. U rows are loaded before the
// first is used.
template <typename TI, typename TO, bool HALF, int U>
__global__ void __launch_bounds__(RT)
    rope_vec_kernel(const __grid_constant__ RopeArgs a, int lanes_log2, int rows_per_y) {
    const int l = threadIdx.x & ((1 << lanes_log2) - 1);
    const long long t =
        static_cast<long long>(blockIdx.x) * (RT >> lanes_log2) + (threadIdx.x >> lanes_log2);
    if (t >= a.tokens) return;
    const int b = static_cast<int>(t) / a.N, n = static_cast<int>(t) - b * a.N;
    const int h0 = blockIdx.y * rows_per_y, h1 = h0 + rows_per_y;
    const long long slot = token_slot(a, t, blockIdx.y == 0 && l == 0);

    constexpr int NP = HALF ? 8 : 4;  // pairs of an item
    constexpr int NC = HALF ? 2 : 1;  // chunks
    const int turns = HALF ? a.rot >> 4 : a.rot >> 3;  // items that are rotated
    const bool turned = l < turns;
    // where the chunks lie; the last one may be missing, and so may the whole item
    const int e0 = HALF && !turned ? a.rot + 16 * (l - turns) : 8 * l;
    const int e1 = !HALF ? 0 : turned ? e0 + a.rot / 2 : e0 + 8;
    if (e0 >= a.d) return;
    const bool second = HALF && e1 < a.d;
    float c[NP], s[NP];
    if (turned && h0 < a.rotated_rows) {
        const int32_t* pos = a.pos + b * a.pos_batch + n;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int pair = NP * l + i;
            turn(a.freqs[pair], axis_pos(a, pos, pair), a.mscale, a.sign, c[i], s[i]);
        }
    }

    for (int gi = 0; gi < a.groups; ++gi) {
        int lo, hi;
        cut(a, gi, h0, h1, lo, hi);
        if (lo >= hi) continue;
        const Rows<TI, TO> r(a, a.g[gi], b, n, slot);
        if (!r.live) continue;
        // ROT: rows are rotated, ALL: every element of them is
        const auto rows = [&](auto ROT, auto ALL) {
            for (int h = lo; h < hi; h += U) {
                Chunk<TI> v[U][NC];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (h + u < hi) {
                        const TI* x = r.x + (h + u) * r.xh;
                        v[u][0].load(x + e0);
                        if (second) v[u][NC - 1].load(x + e1);
                    }
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (h + u < hi) {
                        TO* y = r.y + (h + u) * r.yh;
                        float f[8], g[8];
                        v[u][0].get(f);
                        if (HALF) v[u][NC - 1].get(g);
                        if (ROT && (ALL || turned)) {
#pragma unroll
                            for (int i = 0; i < NP; ++i) {
                                float& p = HALF ? f[i] : f[2 * i & 7];
                                float& q = HALF ? g[i] : f[(2 * i + 1) & 7];
                                const float x0 = p, x1 = q;
                                p = x0 * c[i] - x1 * s[i];
                                q = x1 * c[i] + x0 * s[i];
                            }
                        }
                        put(y + e0, f);
                        if (second) put(y + e1, g);
                    }
            }
        };
        if (!a.g[gi].rotate || a.rot == 0) rows(Const<false>{}, Const<false>{});
        else if (a.rot == a.d) rows(Const<true>{}, Const<true>{});
        else rows(Const<true>{}, Const<false>{});
    }
}

// Any alignment and any even rot: a warp per token, a lane per pair (and per
// element of the rest), one element at a time.
template <typename TI, typename TO>
__global__ void __launch_bounds__(RT)
    rope_scalar_kernel(const __grid_constant__ RopeArgs a, int rows_per_y) {
    const int l = threadIdx.x & 31;
    const long long t = static_cast<long long>(blockIdx.x) * (RT / 32) + (threadIdx.x >> 5);
    if (t >= a.tokens) return;
    const int b = static_cast<int>(t) / a.N, n = static_cast<int>(t) - b * a.N;
    const int h0 = blockIdx.y * rows_per_y, h1 = h0 + rows_per_y;
    const long long slot = token_slot(a, t, blockIdx.y == 0 && l == 0);
    const int pairs = a.rot / 2;
    for (int pair = l; pair < pairs && h0 < a.rotated_rows; pair += 32) {
        float c, s;
        turn(a.freqs[pair], axis_pos(a, a.pos + b * a.pos_batch + n, pair), a.mscale, a.sign, c, s);
        const int e0 = a.half_style ? pair : 2 * pair, e1 = a.half_style ? pair + pairs : 2 * pair + 1;
        for (int gi = 0; gi < a.groups; ++gi) {
            int lo, hi;
            cut(a, gi, h0, h1, lo, hi);
            if (lo >= hi || !a.g[gi].rotate) continue;
            const Rows<TI, TO> r(a, a.g[gi], b, n, slot);
            if (!r.live) continue;
            for (int h = lo; h < hi; ++h) {
                const float f = to_f(r.x[h * r.xh + e0]), g = to_f(r.x[h * r.xh + e1]);
                put1(r.y + h * r.yh + e0, f * c - g * s);
                put1(r.y + h * r.yh + e1, g * c + f * s);
            }
        }
    }
    for (int gi = 0; gi < a.groups; ++gi) {
        int lo, hi;
        cut(a, gi, h0, h1, lo, hi);
        if (lo >= hi) continue;
        const Rows<TI, TO> r(a, a.g[gi], b, n, slot);
        if (!r.live) continue;
        for (int e = (a.g[gi].rotate ? a.rot : 0) + l; e < a.d; e += 32)
            for (int h = lo; h < hi; ++h) put1(r.y + h * r.yh + e, to_f(r.x[h * r.xh + e]));
    }
}

template <typename TI, typename TO>
int launch(const RopeArgs& a, bool vec, cudaStream_t st) {
    // lanes of a token: one per item
    const int need = a.half_style ? (a.d + 15) / 16 : a.d / 8;
    int lanes_log2 = 5;
    vec = vec && need <= RT;
    if (vec)
        for (lanes_log2 = 0; (1 << lanes_log2) < need; ++lanes_log2) {}
    const long long per_cta = RT >> lanes_log2;
    const long long gx = (a.tokens + per_cta - 1) / per_cta;
    if (gx >= (1ll << 31)) return VELOX_EINVAL;
    // The heads are split until there are two CTAs per SM, and no further than four heads
    // a thread, since each part forms its angles again. Queries of a chunk (24 heads of
    // 4608 tokens, bf16): 9.3 us so, 10.9 us with four CTAs per SM; 48 heads of
    // 1000 tokens in the half layout 6.3 and 8.6 us; 200 tokens 3.9 us, 4.4 us down to one head
    const long long want = std::max<long long>(1, (296 + gx - 1) / gx);
    const int parts = static_cast<int>(std::min<long long>({want, (a.rows + 3) / 4, 65535}));
    const int rows_per_y = (a.rows + parts - 1) / parts;
    const dim3 grid(static_cast<unsigned>(gx), (a.rows + rows_per_y - 1) / rows_per_y);
    // rows loaded at once: 128 bytes of a thread (in the half layout and float32 the
    // registers of 64 are what fits)
    constexpr bool F = sizeof(TI) == 4;
    if (!vec)
        rope_scalar_kernel<TI, TO><<<grid, RT, 0, st>>>(a, rows_per_y);
    else if (a.half_style)
        rope_vec_kernel<TI, TO, true, F ? 1 : 4><<<grid, RT, 0, st>>>(a, lanes_log2, rows_per_y);
    else
        rope_vec_kernel<TI, TO, false, F ? 4 : 8><<<grid, RT, 0, st>>>(a, lanes_log2, rows_per_y);
    return cudaGetLastError() == cudaSuccess ? VELOX_OK : VELOX_ECUDA;
}

}  // namespace

int rope_launch(const RopeArgs& a, int in_dtype, bool out_bf16, bool vec, cudaStream_t st) {
    if (in_dtype == VELOX_BF16) return launch<__nv_bfloat16, __nv_bfloat16>(a, vec, st);
    return out_bf16 ? launch<float, __nv_bfloat16>(a, vec, st) : launch<float, float>(a, vec, st);
}

}  // namespace velox
