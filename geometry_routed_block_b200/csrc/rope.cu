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

// The launch overlaps the end of the kernel before this one in the stream, and lets that of
// the next one overlap this one's: nothing in memory is touched before the kernel before
// has ended.
__device__ __forceinline__ void take_turn() {
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

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

__device__ __forceinline__ uint32_t bf2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void unpack(const uint32_t* w, float* f) {  // 8 bf16
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// The 8 elements of an item: SPLIT, 4 at e0 and 4 at e1, else 8 at e0.
template <typename T, bool SPLIT>
struct Item;
template <bool SPLIT>
struct Item<__nv_bfloat16, SPLIT> {
    uint4 r;
    __device__ __forceinline__ void load(const __nv_bfloat16* x, int e0, int e1) {
        if (SPLIT) {
            const uint2 a = *reinterpret_cast<const uint2*>(x + e0);
            const uint2 b = *reinterpret_cast<const uint2*>(x + e1);
            r = make_uint4(a.x, a.y, b.x, b.y);
        } else {
            r = *reinterpret_cast<const uint4*>(x + e0);
        }
    }
    __device__ __forceinline__ void get(float* f) const {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
        unpack(w, f);
    }
};
template <bool SPLIT>
struct Item<float, SPLIT> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* x, int e0, int e1) {
        a = *reinterpret_cast<const float4*>(x + e0);
        b = *reinterpret_cast<const float4*>(x + (SPLIT ? e1 : e0 + 4));
    }
    __device__ __forceinline__ void get(float* f) const {
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
        f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
};
template <bool SPLIT>
__device__ __forceinline__ void put(__nv_bfloat16* y, int e0, int e1, const float* f) {
    const uint4 r = make_uint4(bf2(f[0], f[1]), bf2(f[2], f[3]), bf2(f[4], f[5]), bf2(f[6], f[7]));
    if (SPLIT) {
        *reinterpret_cast<uint2*>(y + e0) = make_uint2(r.x, r.y);
        *reinterpret_cast<uint2*>(y + e1) = make_uint2(r.z, r.w);
    } else {
        *reinterpret_cast<uint4*>(y + e0) = r;
    }
}
template <bool SPLIT>
__device__ __forceinline__ void put(float* y, int e0, int e1, const float* f) {
    *reinterpret_cast<float4*>(y + e0) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(y + (SPLIT ? e1 : e0 + 4)) = make_float4(f[4], f[5], f[6], f[7]);
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

// Whole items of 8 elements, four pairs: interleaved, 8 neighbours; in the half layout
// (SPLIT) 4 neighbours of the first half of the rotated part and the 4 that belong to
// them in the second. 1 << lanes_log2 threads share a token, an item each, and keep its
// factors through all heads. What is not rotated takes the same way past the
// arithmetic, so that a warp does not part. U rows are loaded before the first is
// used.
template <typename TI, typename TO, bool SPLIT, int U>
__global__ void __launch_bounds__(RT)
    rope_vec_kernel(const __grid_constant__ RopeArgs a, int lanes_log2, int rows_per_y) {
    take_turn();
    const int l = threadIdx.x & ((1 << lanes_log2) - 1);
    const long long t =
        static_cast<long long>(blockIdx.x) * (RT >> lanes_log2) + (threadIdx.x >> lanes_log2);
    if (t >= a.tokens || 8 * l >= a.d) return;
    const int b = static_cast<int>(t) / a.N, n = static_cast<int>(t) - b * a.N;
    const int h0 = blockIdx.y * rows_per_y, h1 = h0 + rows_per_y;
    const long long slot = token_slot(a, t, blockIdx.y == 0 && l == 0);

    const bool turned = l < a.rot >> 3;  // the item is rotated
    const int e0 = SPLIT && turned ? 4 * l : 8 * l;
    const int e1 = e0 + (turned ? a.rot >> 1 : 4);
    float c[4], s[4];
    if (turned && h0 < a.rotated_rows) {
        const int32_t* pos = a.pos + b * a.pos_batch + n;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int pair = 4 * l + i;
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
                Item<TI, SPLIT> v[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (h + u < hi) v[u].load(r.x + (h + u) * r.xh, e0, e1);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (h + u < hi) {
                        float f[8];
                        v[u].get(f);
                        if (ROT && (ALL || turned)) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                float& p = f[SPLIT ? i : 2 * i];
                                float& q = f[SPLIT ? i + 4 : 2 * i + 1];
                                const float x0 = p, x1 = q;
                                p = x0 * c[i] - x1 * s[i];
                                q = x1 * c[i] + x0 * s[i];
                            }
                        }
                        put<SPLIT>(r.y + (h + u) * r.yh, e0, e1, f);
                    }
            }
        };
        if (!a.g[gi].rotate || a.rot == 0) rows(Const<false>{}, Const<false>{});
        else if (a.rot == a.d) rows(Const<true>{}, Const<true>{});
        else rows(Const<true>{}, Const<false>{});
    }
}

// The half layout of bf16 rows: an item is 8 neighbours, and the other halves of its
// pairs are an item of another lane of the warp and come from there. Rows are then
// read and written whole, 256 bytes at a time at d = 128: 11.3 us for the queries of a
// chunk, 13.7 us in two times 8 bytes a thread (float32, two times 16 bytes: 16.9 us so,
// 21.5 us exchanged). Each lane of such a couple forms four of their eight angles.
// A warp stays together for the exchange: who has no row only takes part in that.
template <int U>
__global__ void __launch_bounds__(RT, 4)
    rope_half_kernel(const __grid_constant__ RopeArgs a, int lanes_log2, int rows_per_y) {
    using T = __nv_bfloat16;
    take_turn();
    const int l = threadIdx.x & ((1 << lanes_log2) - 1);
    const long long t =
        static_cast<long long>(blockIdx.x) * (RT >> lanes_log2) + (threadIdx.x >> lanes_log2);
    const bool real = t < a.tokens && 8 * l < a.d;
    const int b = real ? static_cast<int>(t) / a.N : 0, n = real ? static_cast<int>(t) - b * a.N : 0;
    const int h0 = blockIdx.y * rows_per_y, h1 = h0 + rows_per_y;
    const long long slot = real ? token_slot(a, t, blockIdx.y == 0 && l == 0) : -1;

    const bool turned = l < a.rot >> 3;
    const int half = a.rot >> 4;  // items of half the rotated part
    const bool first = l < half;
    const int lane = threadIdx.x & 31;
    const int other = !turned ? lane : first ? lane + half : lane - half;
    float c[8], s[8];  // s with the sign of the other half's share
    if (h0 < a.rotated_rows) {
        float cs[4] = {}, sn[4] = {};
        if (real && turned) {
            const int32_t* pos = a.pos + b * a.pos_batch + n;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int pair = first ? 8 * l + i : 8 * (l - half) + 4 + i;
                turn(a.freqs[pair], axis_pos(a, pos, pair), a.mscale, a.sign, cs[i], sn[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float oc = __shfl_sync(~0u, cs[i], other), os = __shfl_sync(~0u, sn[i], other);
            c[i] = first ? cs[i] : oc, c[4 + i] = first ? oc : cs[i];
            s[i] = first ? -sn[i] : os, s[4 + i] = first ? -os : sn[i];
        }
    }

    for (int gi = 0; gi < a.groups; ++gi) {
        int lo, hi;
        cut(a, gi, h0, h1, lo, hi);
        if (lo >= hi) continue;
        const Rows<T, T> r(a, a.g[gi], b, n, slot);
        const bool live = real && r.live;
        const T* x = r.x + 8 * l;
        T* y = r.y + 8 * l;
        const bool rotate = a.g[gi].rotate;
        for (int h = lo; h < hi; h += U) {
            uint4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                v[u] = make_uint4(0, 0, 0, 0);
                if (live && h + u < hi) v[u] = *reinterpret_cast<const uint4*>(x + (h + u) * r.xh);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (rotate) {
                    const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
                    uint32_t q[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) q[i] = __shfl_sync(~0u, w[i], other);
                    if (turned) {
                        float f[8], g[8];
                        unpack(w, f);
                        unpack(q, g);
#pragma unroll
                        for (int i = 0; i < 8; ++i) f[i] = f[i] * c[i] + g[i] * s[i];
                        v[u] = make_uint4(bf2(f[0], f[1]), bf2(f[2], f[3]), bf2(f[4], f[5]),
                                          bf2(f[6], f[7]));
                    }
                }
                if (live && h + u < hi) *reinterpret_cast<uint4*>(y + (h + u) * r.yh) = v[u];
            }
        }
    }
}

// Any alignment and any even rot: a warp per token, a lane per pair (and per
// element of the rest), one element at a time.
template <typename TI, typename TO>
__global__ void __launch_bounds__(RT)
    rope_scalar_kernel(const __grid_constant__ RopeArgs a, int rows_per_y) {
    take_turn();
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
    int lanes_log2 = 5;
    vec = vec && a.d / 8 <= RT;
    if (vec)
        for (lanes_log2 = 0; (1 << lanes_log2) < a.d / 8; ++lanes_log2) {}
    const long long per_cta = RT >> lanes_log2;
    const long long gx = (a.tokens + per_cta - 1) / per_cta;
    if (gx >= (1ll << 31)) return VELOX_EINVAL;
    // The heads are split until there are two CTAs per SM, and no further than four heads
    // a thread, since each part forms its angles again. Queries of a chunk (24 heads of
    // 4608 tokens, bf16): 9.3 us so, 10.6 us with four CTAs per SM (half layout 11.3 and 12.3);
    // 64 tokens of 72 heads 2.9 us, 3.5 us split to two heads
    const long long want = std::max<long long>(1, (296 + gx - 1) / gx);
    const int parts = static_cast<int>(std::min<long long>({want, (a.rows + 3) / 4, 65535}));
    const int rows_per_y = (a.rows + parts - 1) / parts;
    const dim3 grid(static_cast<unsigned>(gx), (a.rows + rows_per_y - 1) / rows_per_y);
    constexpr bool BF = sizeof(TI) == 2;
    constexpr int U = BF ? 8 : 4;  // rows at once: 128 bytes of a thread
    // in the half layout an item's other half is a whole item, in the same warp
    const bool exchange = BF && a.rot > 0 && a.rot % 16 == 0 && a.d <= 256;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(RT);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t rc =
        !vec ? cudaLaunchKernelEx(&cfg, rope_scalar_kernel<TI, TO>, a, rows_per_y)
        : !a.half_style
            ? cudaLaunchKernelEx(&cfg, rope_vec_kernel<TI, TO, false, U>, a, lanes_log2, rows_per_y)
        : exchange ? cudaLaunchKernelEx(&cfg, rope_half_kernel<4>, a, lanes_log2, rows_per_y)
                   : cudaLaunchKernelEx(&cfg, rope_vec_kernel<TI, TO, true, U>, a, lanes_log2, rows_per_y);
    return rc == cudaSuccess ? VELOX_OK : VELOX_ECUDA;
}

}  // namespace

int rope_launch(const RopeArgs& a, int in_dtype, bool out_bf16, bool vec, cudaStream_t st) {
    if (in_dtype == VELOX_BF16) return launch<__nv_bfloat16, __nv_bfloat16>(a, vec, st);
    return out_bf16 ? launch<float, __nv_bfloat16>(a, vec, st) : launch<float, float>(a, vec, st);
}

}  // namespace velox
