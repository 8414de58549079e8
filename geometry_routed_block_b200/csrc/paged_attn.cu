// Attention of one new token per request over a paged KV cache, split over the
// length and joined.
//
// Mathematics: for query head h of request r and its n = lens[r] keys
//   s_j = scale q.k_j,  o = sum_j 2^(s'_j - m) v_j / sum_j 2^(s'_j - m),
// s' = s log2(e), m the running maximum; parts of the history with their own
// (m, l, o) are joined by o = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i.
//
// What bounds it: bytes. Every key and value is read once and used by the query
// heads that share it, 2 H / Hkv FLOP per byte: far below the tensor cores'
// rate, so the products run on warp-level matrix instructions, whose 16 rows
// suit the few query heads (a 128-row tile would be padding), and everything
// else serves the stream of loads:
//   - The history is cut in units of 16 tokens (K and V of one key head: 8 KB at
//     d = 128). Units of all (request, key head, tile of query heads) rows are
//     numbered in order, and every CTA takes an equal, contiguous share, whatever
//     the lengths are; no length is read by the host. A CTA's share covers the
//     end of one row, whole rows, and the beginning of another. Whole rows are
//     finished here, the others leave (m, l, o) in the workspace, two at most
//     per CTA, and a second kernel joins them.
//   - Within a CTA, units go to the warps in turn. A warp runs alone: it
//     fetches its units by TMA into its own ring of shared memory (128-byte
//     swizzle), several units ahead and across row ends, and needs no other warp
//     until the row ends, where the warps' (m, l, o) meet in shared memory.
//   - S = Q K^T has the query heads in rows 0-7 (and heads 8-15 in rows 8-15, when
//     more than 8 share a key head). P is split into two bf16, P = hi + lo, with
//     hi in rows 0-7 and lo in rows 8-15 of one product with V: the rows that 8
//     heads leave free carry the second half, so that P keeps 16 bits at no cost.
//     A lo row that met an infinite value (inf - inf) is left out at the end.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "attn_common.cuh"

namespace velox {

namespace {

constexpr int UNIT = 16;       // tokens per unit: the smallest page
constexpr int NW = 4;          // warps per CTA
constexpr int NT = NW * 32;
constexpr int MAX_GRID = 320;  // CTAs at most (two per SM)
// units per CTA at least: a share of fewer would leave warps without work and cost more
// joining than it saves
constexpr int MIN_SHARE = 2 * NW;

template <int D, int MT>
struct Cfg {
    static constexpr int HEADS = 8 * MT;           // query heads per tile
    static constexpr int HALF = UNIT * 128;        // 16 tokens x 64 columns
    static constexpr int TILE = UNIT * D * 2;      // K or V of a unit
    static constexpr int STAGE = 2 * TILE;
    static constexpr int ST = D == 128 ? 3 : 6;    // ring depth per warp
    static constexpr int OFF_O = NW * ST * STAGE;  // float [NW][8][D]
    static constexpr int OFF_M = OFF_O + NW * 8 * D * 4;    // float [NW][HEADS]
    static constexpr int OFF_L = OFF_M + NW * HEADS * 4;    // float [NW][HEADS]
    static constexpr int OFF_BAR = OFF_L + NW * HEADS * 4;  // uint64 [NW][ST]
    static constexpr int OFF_SH = OFF_BAR + NW * ST * 8;    // int64 [NW + 4]
    static constexpr int OFF_ABORT = OFF_SH + (NW + 4) * 8;
    static constexpr int SMEM = OFF_ABORT + 8;
    static constexpr int PART = HEADS * (D + 2);   // floats of a partial result: o, m, l
};

__device__ __forceinline__ int clamp_len(int n, int cap) { return min(max(n, 0), cap); }
__device__ __forceinline__ int units_of(int n) { return (n + UNIT - 1) / UNIT; }

// Where the work lies: total units, and the row that holds a given unit.
struct Place {
    long long total;
    int grid;       // CTAs that take a share
    int r, row, u;  // request, row in it (key head x head tile), unit in the row
    int n, units;   // tokens and units of the request
    long long base; // first unit of the row
};

__device__ __forceinline__ long long share(long long total, int grid, int c) {
    return total * c / grid;
}

// Every thread of the CTA calls it. Unit number of share `c` -> place (c = grid:
// only total and grid are set). sh: at least NT + 8 long longs.
__device__ __forceinline__ void locate(const PagedAttnArgs& a, int c, Place& p, long long* sh,
                                       bool report) {
    const int rows = a.Hkv * a.head_tiles, cap = a.max_pages * a.page;
    const int per = (a.R + NT - 1) / NT;
    const int r0 = min(a.R, static_cast<int>(threadIdx.x) * per), r1 = min(a.R, r0 + per);
    long long mine = 0;
    bool bad = false;
    for (int r = r0; r < r1; ++r) {
        const int n = a.lens[r];
        bad |= n < 0 || n > cap;
        mine += units_of(clamp_len(n, cap));
    }
    if (report && bad && a.status) atomicOr(a.status, VELOX_STATUS_BAD_INDEX);
    long long x = mine;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(~0u, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sh[warp] = x;
    __syncthreads();
    long long before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        if (w < warp) before += sh[w];
        total += sh[w];
    }
    long long first = before + x - mine;  // units of the requests before r0 (one row each)
    p.total = total * rows;
    const long long most = (p.total + MIN_SHARE - 1) / MIN_SHARE;
    p.grid = static_cast<int>(min(static_cast<long long>(a.grid), max(most, 1ll)));
    if (c < p.grid && p.total > 0) {
        const long long s = share(p.total, p.grid, c);
        if (s >= first * rows && s < (first + mine) * rows) {
            int r = r0;
            for (; r < r1; ++r) {
                const int un = units_of(clamp_len(a.lens[r], cap));
                if (s < (first + un) * rows) break;
                first += un;
            }
            const int n = clamp_len(a.lens[r], cap), un = units_of(n);
            const long long in = s - first * rows;
            const int row = static_cast<int>(in / un);
            sh[NW] = r;
            sh[NW + 1] = row;
            sh[NW + 2] = n;
            sh[NW + 3] = s - (in - static_cast<long long>(row) * un);
        }
        __syncthreads();
        p.r = static_cast<int>(sh[NW]);
        p.row = static_cast<int>(sh[NW + 1]);
        p.n = static_cast<int>(sh[NW + 2]);
        p.units = units_of(p.n);
        p.base = sh[NW + 3];
        p.u = static_cast<int>(s - p.base);
    }
}

// the next row that has units, after the one at p (which exists: the caller knows
// that units are left)
__device__ __forceinline__ void next_row(const PagedAttnArgs& a, Place& p) {
    const int rows = a.Hkv * a.head_tiles, cap = a.max_pages * a.page;
    p.base += p.units;
    p.u = 0;
    if (++p.row < rows) return;
    p.row = 0;
    do {
        ++p.r;
        p.n = p.r < a.R ? clamp_len(a.lens[p.r], cap) : UNIT;
    } while (p.n == 0);
    p.units = units_of(p.n);
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// byte of 16-byte chunk `c` (of D/8) of token `row` in a K or V tile: halves of 64
// columns, 128-byte rows, chunks swizzled by the row
template <int D, int MT>
__device__ __forceinline__ uint32_t tile_at(int row, int c) {
    return (c >> 3) * Cfg<D, MT>::HALF + row * 128 + (((c & 7) ^ (row & 7)) << 4);
}

__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }

template <int D, int MT>
__global__ void __launch_bounds__(NT, 2)
    paged_attn_kernel(const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ PagedAttnArgs a) {
    using C = Cfg<D, MT>;
    // the swizzle counts rows from 1024-byte boundaries; there is no static
    // shared memory in front, and no room for slack with two CTAs per SM
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    long long* sh = reinterpret_cast<long long*>(smem + C::OFF_SH);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t ring = sbase + warp * C::ST * C::STAGE;
    const uint32_t bars = sbase + C::OFF_BAR + warp * C::ST * 8;
    const int rows = a.Hkv * a.head_tiles, cap = a.max_pages * a.page;

    // lets the joining kernel's CTAs settle on the SMs; they wait for this grid's end
    asm volatile("griddepcontrol.launch_dependents;");
    if (threadIdx.x == 0) {
        *abort_flag = 0;
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
    }
    if (lane == 0)
        for (int s = 0; s < C::ST; ++s) mbar_init(bars + 8 * s, 1);
    fence_mbar_init();

    // requests without tokens get zeros
    const int row_elems = a.H * D;
    for (int r = blockIdx.x; r < a.R; r += gridDim.x) {
        if (clamp_len(a.lens[r], cap) > 0) continue;
        for (int i = threadIdx.x; i < row_elems / 8; i += NT)
            reinterpret_cast<uint4*>(a.o + static_cast<long long>(r) * row_elems)[i] =
                make_uint4(0, 0, 0, 0);
        if (a.lse)
            for (int h = threadIdx.x; h < a.H; h += NT)
                a.lse[static_cast<long long>(r) * a.H + h] = -INFINITY;
    }

    Place p;
    const int cta = blockIdx.x;
    locate(a, cta, p, sh, cta == 0);
    __syncthreads();  // barriers initialised
    if (cta >= p.grid || p.total == 0) return;
    const long long s0 = share(p.total, p.grid, cta), s1 = share(p.total, p.grid, cta + 1);
    if (s0 >= s1) return;

    // ---- this warp's loads: units s0 + warp, + NW, ... of the CTA's share
    Place f = p;                   // row of the next unit to fetch
    long long fg = s0 + warp;      // its number
    int page_id = 0, page_row = 0; // its page, looked up one unit ahead
    auto find = [&]() {            // moves f to unit fg and looks its page up
        if (fg >= s1) return;
        while (fg >= f.base + f.units) next_row(a, f);
        const int tok = static_cast<int>(fg - f.base) * UNIT;
        page_row = tok & (a.page - 1);
        page_id = a.table[static_cast<long long>(f.r) * a.max_pages + tok / a.page];
    };
    int f_head = 0;
    auto fetch = [&](int slot) {  // lane 0 fetches unit fg into `slot`
        if (lane == 0) {
            int id = page_id;
            if (id < 0 || id >= a.num_pages) {
                if (a.status) atomicOr(a.status, VELOX_STATUS_BAD_INDEX);
                id = 0;
            }
            f_head = f.row / a.head_tiles;
            const int y = (id * a.Hkv + f_head) * a.page + page_row;
            const uint32_t bar = bars + 8 * slot, dst = ring + slot * C::STAGE;
            mbar_arrive_expect_tx(bar, C::STAGE);
#pragma unroll
            for (int h = 0; h < D / 64; ++h) tma_load_2d(dst + h * C::HALF, &tmK, bar, 64 * h, y);
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
                tma_load_2d(dst + C::TILE + h * C::HALF, &tmV, bar, 64 * h, y);
        }
        fg += NW;
        find();
    };
    find();
    int issued = 0;  // units fetched so far, modulo nothing: counts up
    for (int s = 0; s < C::ST; ++s)
        if (fg < s1) {
            fetch(s);
            ++issued;
        }

    const int g = lane >> 2, t = lane & 3;
    int done = 0, slot = 0;
    uint32_t parity = 0;
    bool ok = true;
    long long cg = s0 + warp;  // this warp's next unit
    for (long long at = s0; at < s1;) {
        const long long row_end = min(p.base + p.units, s1);
        const int hk = p.row / a.head_tiles, ht = p.row - hk * a.head_tiles;
        const int head0 = hk * a.group + ht * a.tile_heads;
        const int heads = min(a.tile_heads, a.group - ht * a.tile_heads);
        const long long q_row = static_cast<long long>(p.r) * a.H + head0;

        float o[MT][D / 8][4];
        float m[MT], l[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            m[i] = -INFINITY, l[i] = 0.0f;
#pragma unroll
            for (int j = 0; j < D / 8; ++j) o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.0f;
        }
        if (cg < row_end) {
            uint32_t q[MT][D / 16][2];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const bool have = 8 * i + g < heads;
                const uint32_t* src =
                    reinterpret_cast<const uint32_t*>(a.q + (q_row + (have ? 8 * i + g : 0)) * D) + t;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    q[i][k][0] = have ? src[8 * k] : 0u;
                    q[i][k][1] = have ? src[8 * k + 4] : 0u;
                }
            }
            for (; cg < row_end; cg += NW) {
                ok = ok && mbar_wait(bars + 8 * slot, parity, abort_flag, a.wait_ns);
                ok = __all_sync(~0u, ok);
                if (!ok) break;
                const uint32_t kt = ring + slot * C::STAGE, vt = kt + C::TILE;
                const int valid = p.n - static_cast<int>(cg - p.base) * UNIT;  // tokens left
                if (valid < UNIT) {
                    // values behind the last token may be anything: their weight is 0, but
                    // 0 * NaN is not
                    for (int i = lane; i < (UNIT - valid) * (D / 8); i += 32)
                        *reinterpret_cast<uint4*>(smem + (vt - sbase) +
                                                  tile_at<D, MT>(valid + i / (D / 8), i % (D / 8))) =
                            make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();  // before the next fetch into this slot
                    __syncwarp();
                }
                // S: two key groups of 8, each in two chains over d
                float s[2][2][4];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) s[i][j][0] = s[i][j][1] = s[i][j][2] = s[i][j][3] = 0.0f;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    uint32_t b[4];  // keys 0-7: d lo, d hi; keys 8-15: d lo, d hi
                    ldsm4(kt + tile_at<D, MT>((lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)),
                          b);
                    const uint32_t a1 = MT == 2 ? q[MT - 1][k][0] : 0u;
                    const uint32_t a3 = MT == 2 ? q[MT - 1][k][1] : 0u;
                    mma16816(s[k & 1][0], q[0][k][0], a1, q[0][k][1], a3, b[0], b[1]);
                    mma16816(s[k & 1][1], q[0][k][0], a1, q[0][k][1], a3, b[2], b[3]);
                }
                uint32_t hi[MT][2], lo[MT][2];
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    float x[4];  // keys 2t, 2t+1, 8+2t, 8+2t+1 of head 8 i + g
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        x[j] = (s[0][j >> 1][2 * i + (j & 1)] + s[1][j >> 1][2 * i + (j & 1)]) *
                               a.scale_log2;
                        if (8 * (j >> 1) + 2 * t + (j & 1) >= valid) x[j] = -INFINITY;
                    }
                    float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
                    const float m_new = fmaxf(m[i], top);
                    if (__any_sync(~0u, m_new > m[i])) {
                        // m = -inf: nothing has been summed yet, and 2^(-inf) = 0
                        const float scale = m_new == -INFINITY ? 1.0f : ex2_approx(m[i] - m_new);
                        l[i] *= scale;
#pragma unroll
                        for (int j = 0; j < D / 8; ++j) {
                            o[i][j][0] *= scale, o[i][j][1] *= scale;
                            o[i][j][2] *= scale, o[i][j][3] *= scale;
                        }
                        m[i] = m_new;
                    }
                    const float ref = m[i] == -INFINITY ? 0.0f : m[i];
                    float pr[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) pr[j] = ex2_approx(x[j] - ref);
                    l[i] += (pr[0] + pr[1]) + (pr[2] + pr[3]);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        hi[i][j] = pack_bf16x2(pr[2 * j], pr[2 * j + 1]);
                        lo[i][j] = pack_bf16x2(pr[2 * j] - bf16_lo(hi[i][j]),
                                               pr[2 * j + 1] - bf16_hi(hi[i][j]));
                    }
                }
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    uint32_t b[4];  // d 16 j .. +7: keys lo, keys hi; the next 8: keys lo, keys hi
                    ldsm4_t(vt + tile_at<D, MT>((lane & 7) + (((lane >> 3) & 1) << 3),
                                                2 * j + (lane >> 4)),
                            b);
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        mma16816(o[i][2 * j], hi[i][0], lo[i][0], hi[i][1], lo[i][1], b[0], b[1]);
                        mma16816(o[i][2 * j + 1], hi[i][0], lo[i][0], hi[i][1], lo[i][1], b[2], b[3]);
                    }
                }
                __syncwarp();  // every lane has read the slot
                ++done;
                if (fg < s1) {
                    fetch(slot);
                    ++issued;
                }
                if (++slot == C::ST) slot = 0, parity ^= 1;
            }
        }
        // ---- the row (or this CTA's part of it) is done: join the warps
        float* sm_o = reinterpret_cast<float*>(smem + C::OFF_O);
        float* sm_m = reinterpret_cast<float*>(smem + C::OFF_M);
        float* sm_l = reinterpret_cast<float*>(smem + C::OFF_L);
        const bool whole = at == p.base && row_end == p.base + p.units;
        float* part = a.part + static_cast<long long>(2 * cta + (at == s0 ? 0 : 1)) * C::PART;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            l[i] += __shfl_xor_sync(~0u, l[i], 1);
            l[i] += __shfl_xor_sync(~0u, l[i], 2);
            if (t == 0) sm_m[warp * C::HEADS + 8 * i + g] = m[i], sm_l[warp * C::HEADS + 8 * i + g] = l[i];
            if (8 * i + g < heads) {
#pragma unroll
                for (int j = 0; j < D / 8; ++j) {
                    float v0 = o[i][j][0], v1 = o[i][j][1];
                    if (isfinite(o[i][j][2])) v0 += o[i][j][2];
                    if (isfinite(o[i][j][3])) v1 += o[i][j][3];
                    *reinterpret_cast<float2*>(sm_o + (warp * 8 + g) * D + 8 * j + 2 * t) =
                        make_float2(v0, v1);
                }
            }
            __syncthreads();
            for (int e = threadIdx.x; e < 8 * D; e += NT) {
                const int h = e / D, col = e % D, hh = 8 * i + h;
                if (hh >= heads) break;
                float top = sm_m[hh];
#pragma unroll
                for (int w = 1; w < NW; ++w) top = fmaxf(top, sm_m[w * C::HEADS + hh]);
                const float ref = top == -INFINITY ? 0.0f : top;
                float sum = 0.0f, acc = 0.0f;
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    const float x = ex2_approx(sm_m[w * C::HEADS + hh] - ref);
                    sum += x * sm_l[w * C::HEADS + hh];
                    // a warp without units has m = -inf and o = 0
                    acc += x * sm_o[(w * 8 + h) * D + col];
                }
                if (whole) {
                    a.o[(q_row + hh) * D + col] = __float2bfloat16_rn(acc / sum);
                    if (a.lse && col == 0)
                        a.lse[q_row + hh] = (ref + log2f(sum)) * 0.6931471805599453f;
                } else {
                    part[hh * D + col] = acc;
                    if (col == 0) {
                        part[C::HEADS * D + hh] = top;
                        part[C::HEADS * D + C::HEADS + hh] = sum;
                    }
                }
            }
            __syncthreads();
        }
        at = row_end;
        if (at < s1) next_row(a, p);
    }
    // a wait that ran out: what is still in flight lands before the CTA leaves
    if (!ok) {
        if (lane == 0 && a.status) atomicOr(a.status, VELOX_STATUS_TIMEOUT);
        volatile int never = 0;
        for (; done < issued; ++done) {
            if (!mbar_wait(bars + 8 * slot, parity, &never, a.wait_ns)) break;
            if (++slot == C::ST) slot = 0, parity ^= 1;
        }
    }
}

// Joins the parts of the rows that more than one CTA worked on. CTA (c, head):
// if share c is the first to begin inside a row that an earlier share began, it
// joins that row's query head. A row's parts are those of consecutive shares; the
// order of the sums is fixed.
template <int D, int MT>
__global__ void __launch_bounds__(NT)
    paged_join_kernel(const __grid_constant__ PagedAttnArgs a) {
    using C = Cfg<D, MT>;
    __shared__ long long sh[NW + 4];
    __shared__ float red_m[NW], red_l[NW], red_o[NW][D];
    Place p;
    const int c = blockIdx.x + 1, hh = blockIdx.y;
    locate(a, c, p, sh, false);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (c >= p.grid || p.total == 0) return;
    const long long s = share(p.total, p.grid, c);
    // a share before this one began the row, and none but that one lies before
    if (s == p.base || share(p.total, p.grid, c - 1) > p.base) return;
    const int hk = p.row / a.head_tiles, ht = p.row - hk * a.head_tiles;
    const int heads = min(a.tile_heads, a.group - ht * a.tile_heads);
    if (hh >= heads) return;
    const long long end = p.base + p.units;
    // the last share that begins before the row's end
    const int last = static_cast<int>((end * p.grid - 1) / p.total);
    const int first = c - 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int PER = D / 32;

    float top = -INFINITY, sum = 0.0f, acc[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = 0.0f;
    for (int i = first + warp; i <= last; i += NW) {
        // a share's first row is its part 0
        const int which = 2 * i + (share(p.total, p.grid, i) >= p.base ? 0 : 1);
        const float* part = a.part + static_cast<long long>(which) * C::PART;
        const float m = part[C::HEADS * D + hh], l = part[C::HEADS * D + C::HEADS + hh];
        float v[PER];
#pragma unroll
        for (int e = 0; e < PER; ++e) v[e] = part[hh * D + lane + 32 * e];
        const float m_new = fmaxf(top, m);
        const float ref = m_new == -INFINITY ? 0.0f : m_new;
        const float x = ex2_approx(top - ref), y = ex2_approx(m - ref);
        sum = sum * x + l * y;
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[e] = acc[e] * x + v[e] * y;
        top = m_new;
    }
    if (lane == 0) red_m[warp] = top, red_l[warp] = sum;
#pragma unroll
    for (int e = 0; e < PER; ++e) red_o[warp][lane + 32 * e] = acc[e];
    __syncthreads();
    if (threadIdx.x < D) {
        float m = red_m[0];
#pragma unroll
        for (int w = 1; w < NW; ++w) m = fmaxf(m, red_m[w]);
        const float ref = m == -INFINITY ? 0.0f : m;
        float l = 0.0f, o = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float x = ex2_approx(red_m[w] - ref);
            l += x * red_l[w];
            o += x * red_o[w][threadIdx.x];
        }
        const long long row =
            static_cast<long long>(p.r) * a.H + hk * a.group + ht * a.tile_heads + hh;
        a.o[row * D + threadIdx.x] = __float2bfloat16_rn(o / l);
        if (a.lse && threadIdx.x == 0) a.lse[row] = (ref + log2f(l)) * 0.6931471805599453f;
    }
}

template <int D, int MT>
int launch(const void* k_pages, const void* v_pages, PagedAttnArgs a, cudaStream_t st) {
    using C = Cfg<D, MT>;
    static_assert(C::SMEM + 1024 <= 233472 / 2, "shared memory of two CTAs");
    static_assert(C::HALF % 1024 == 0, "swizzle atoms");
    CUtensorMap tk, tv;
    const uint64_t pool = static_cast<uint64_t>(a.num_pages) * a.Hkv * a.page;
    if (!make_tmap(&tk, k_pages, pool, D, UNIT) || !make_tmap(&tv, v_pages, pool, D, UNIT))
        return VELOX_ECUDA;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return VELOX_ECUDA;
    a.grid = std::min(2 * sms, MAX_GRID);
    auto kern = paged_attn_kernel<D, MT>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) !=
        cudaSuccess)
        return VELOX_ECUDA;
    kern<<<a.grid, NT, C::SMEM, st>>>(tk, tv, a);
    if (cudaGetLastError() != cudaSuccess) return VELOX_ECUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(a.grid - 1, a.tile_heads);
    cfg.blockDim = dim3(NT);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_join_kernel<D, MT>, a) == cudaSuccess ? VELOX_OK
                                                                               : VELOX_ECUDA;
}

}  // namespace

size_t paged_attn_ws_bytes(int R, int H, int Hkv, int d) {
    const int mt = H / Hkv > 8 ? 2 : 1;
    return static_cast<size_t>(2 * MAX_GRID) * 8 * mt * (d + 2) * sizeof(float);
}

int paged_attn_launch(const void* k_pages, const void* v_pages, const PagedAttnArgs& args, int d,
                      cudaStream_t st) {
    PagedAttnArgs a = args;
    a.group = a.H / a.Hkv;
    a.head_tiles = (a.group + 15) / 16;
    a.tile_heads = (a.group + a.head_tiles - 1) / a.head_tiles;
    const bool wide = a.group > 8;
    if (d == 128)
        return wide ? launch<128, 2>(k_pages, v_pages, a, st) : launch<128, 1>(k_pages, v_pages, a, st);
    return wide ? launch<64, 2>(k_pages, v_pages, a, st) : launch<64, 1>(k_pages, v_pages, a, st);
}

}  // namespace velox
