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
//   - The history is cut in units of 8 KB (K and V of one key head: 16 tokens at d = 128, 32
//     at d = 64). The units of all (request, key head, tile of query heads) rows are
//     numbered in order, with ROW_COST empty units behind each row for what a
//     row costs beyond its units, and every warp takes an equal, contiguous share,
//     whatever the lengths are; no length is read by the host. Rows that lie
//     inside a share, the many short ones, are finished by their warp alone.
//   - A warp fetches its units by TMA into its own ring of shared memory (128-byte
//     swizzle), several units ahead and across row ends, and waits for no other
//     warp until its share is done. Then the CTA joins the parts of rows that its
//     warps share, through shared memory; what reaches beyond the CTA (two rows
//     at most) goes as (m, l, o) to the workspace, and a second kernel joins that.
//   - Rows of short histories (by the table's width), and those of a single request, which
//     are all of one length, are not dealt out: a CTA or a cluster of CTAs takes a row, and
//     joins it through distributed shared memory, in one launch.
//   - S = Q K^T has the query heads in rows 0-7 (and heads 8-15 in rows 8-15, when
//     more than 8 share a key head). P is split into two bf16, P = hi + lo, with
//     hi in rows 0-7 and lo in rows 8-15 of one product with V: the rows that 8
//     heads leave free carry the second half, so that P keeps 16 bits at no cost.
//     A lo row that met an infinite value (inf - inf) is left out at the end.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "attn_common.cuh"

namespace velox {

namespace {

constexpr int BOX = 16;        // tokens that one load fetches: the smallest page
constexpr int NW = 4;          // warps per CTA
constexpr int NT = NW * 32;
constexpr int MAX_GRID = 320;  // CTAs at most
// Bytes that the CTAs together keep in flight, in whole units a warp. More is slower, DRAM then
// serves too many places at once: the whole history of 24 heads (2.77 GB, clusters of 10) takes
// 394 us with two units a warp (15.7 MB) and 427 with three (23.6 MB), in a steady loop under
// the power cap 404 and 413; a ragged batch of 64 requests 78.4 (17.0 MB) and 81.9 (25.5 MB)
constexpr double IN_FLIGHT = 17.5e6;
constexpr int JT = 256;        // threads of the joining kernel
constexpr int JW = JT / 32;
constexpr int PPL = (MAX_GRID + JT - 1) / JT;  // parts that a lane looks after
constexpr int ROW_COST = 2;    // empty units that a row counts for
// units per warp at least: fewer would cost more joining than they save
constexpr int MIN_SHARE = 2;

// Where no row can be longer (by the width of the table) than so many tokens for each of the
// n = 1, 2, 4 or 8 CTAs that every row can have at once, rows are not dealt out by length:
// a CTA or a cluster takes a row, in one launch and without a workspace. 32 / 8 heads, one
// request, history in L2: 20 tokens 4.4 us (dealt out 6.9), 257 tokens 6.0 (one CTA a row 8.0,
// dealt out 9.5), 480 tokens 6.4 (10.1, 8.9), 1024 tokens 7.2 (16.3, 8.9).
constexpr int WHOLE_TOKENS = 512, WHOLE_CTAS = 256;

template <int D, int MT>
struct Cfg {
    static constexpr int HEADS = 8 * MT;           // query heads per tile
    static constexpr int SUB = 128 / D;            // boxes of 16 tokens in a unit
    static constexpr int UNIT = SUB * BOX;         // tokens of a unit: 8 KB of K and V
    static constexpr int HALF = BOX * 128;         // a box: 16 tokens x 64 columns
    static constexpr int TILE = UNIT * D * 2;      // K or V of a unit
    static constexpr int STAGE = 2 * TILE;
    // units that a warp's ring has room for with two CTAs per SM (the launch may use fewer)
    static constexpr int ST = MT == 2 ? 2 : 3;
    static constexpr int OFF_O = NW * ST * STAGE;  // float [NW][HEADS][D]: a warp's first row
    static constexpr int OFF_M = OFF_O + NW * HEADS * D * 4;   // float [2 NW][HEADS]
    static constexpr int OFF_L = OFF_M + 2 * NW * HEADS * 4;   // float [2 NW][HEADS]
    static constexpr int OFF_SH = OFF_L + 2 * NW * HEADS * 4;  // int64 [NW][6]: shares' rows
    static constexpr int OFF_BAR = OFF_SH + NW * 6 * 8;        // uint64 [NW][ST]
    static constexpr int OFF_ENT = OFF_BAR + NW * ST * 8;      // int [2 NW][4]: the parts
    static constexpr int OFF_ABORT = OFF_ENT + 2 * NW * 16;
    static constexpr int SMEM = OFF_ABORT + 8;
    static_assert(ST * STAGE >= HEADS * D * 4, "a warp's last row takes its ring's place");
    static constexpr int PART = HEADS * (D + 2);   // floats of a partial result: o, m, l
};

__device__ __forceinline__ int clamp_len(int n, int cap) { return min(max(n, 0), cap); }
template <int D>
__device__ __forceinline__ int units_of(int n) {
    constexpr int UNIT = Cfg<D, 1>::UNIT;
    return n / UNIT + (n % UNIT != 0);
}

// A row: one key head (and tile of its query heads) of one request. Its real units
// are base .. base + units - 1 in the numbering of all, ROW_COST empty ones follow.
struct Row {
    long long base;
    int r, row;     // request, row in it
    int n, units;   // tokens and units of the request
};
// The total (the empty units included) in equal shares, NW to a CTA: `more` of each
// + 1 units, then of `each`.
struct Work {
    long long total, each;
    int grid;  // CTAs that take a share
    int more;
    // where warp share w begins
    __device__ __forceinline__ long long start(int w) const { return w * each + min(w, more); }
    // the CTA in whose share unit u lies
    __device__ __forceinline__ int cta_of(long long u) const;
};

// 64-bit division, 32-bit wherever the numbers are: several of the former are what
// a short call would spend most of its time on
__device__ __forceinline__ long long quotient(long long x, long long d) {
    if (((x | d) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(d);
    return x / d;
}

__device__ __forceinline__ int Work::cta_of(long long u) const {
    u = min(u, total - 1);
    const long long first = more * (each + 1);
    const long long w = u < first ? quotient(u, each + 1) : more + quotient(u - first, each);
    return static_cast<int>(w) / NW;
}

__device__ __forceinline__ int weight(int units) { return units > 0 ? units + ROW_COST : 0; }

// The row of q and o that request r attends with: its own number or, in a plan's STEP, that
// of its last new token, -1 where it has none (`bad`: where there can be no such row). An idle
// request counts as one without tokens: 64 ragged requests take 88 us, 58 with every second
// one idle, 13 with 7 of 8. STEP is a parameter of the kernels: asked at run time it cost
// calls without a plan 0.1 to 0.4 us.
template <bool STEP>
__device__ __forceinline__ int token_row(const PagedAttnArgs& a, int r, bool& bad) {
    if (!STEP) return r;
    const int begin = a.cu[r], end = a.cu[r + 1];
    const bool there = begin >= 0 && begin < end && end <= a.N;
    bad |= !there && begin != end;
    return there ? end - 1 : -1;
}
// the same for a request that has one (within q, should cu change meanwhile)
template <bool STEP>
__device__ __forceinline__ int row_of(const PagedAttnArgs& a, int r) {
    return STEP ? min(max(a.cu[r + 1] - 1, 0), a.N - 1) : r;
}
// the tokens that request r attends to: none where it has no row
template <bool STEP>
__device__ __forceinline__ int tokens_of(const PagedAttnArgs& a, int r, int cap) {
    bool bad = false;
    return token_row<STEP>(a, r, bad) < 0 ? 0 : clamp_len(a.lens[r], cap);
}

// Every thread of the CTA calls it. Counts the work, and finds the rows in which
// `count` warp shares begin, those numbered first, first + step, ...: sh[6 i] onwards
// gets the i-th's row (nothing where there is no such share, or an empty one at the
// end). sh: 6 long longs per share, and one per warp at least. The caller lets the
// CTA meet before it reads sh. Lengths beyond KEPT a thread are looked at twice: should one
// change meanwhile, what is found is meaningless, but lies within the arguments.
template <int D, bool STEP, int THREADS>
__device__ __forceinline__ Work locate(const PagedAttnArgs& a, int first, int count, int step,
                                       long long* sh, bool report) {
    const int rows = a.Hkv * a.head_tiles, cap = a.max_pages * a.page;
    const int each = (a.R + THREADS - 1) / THREADS;
    const int r0 = min(a.R, static_cast<int>(threadIdx.x) * each), r1 = min(a.R, r0 + each);
    long long mine = 0;
    bool bad = false;
    constexpr int KEPT = 4;  // lengths held in registers: a second look costs as much as the first
    int kept[KEPT] = {};
#pragma unroll
    for (int i = 0; i < KEPT; ++i)
        if (r0 + i < r1) kept[i] = a.lens[r0 + i];
    if (STEP)
#pragma unroll
        for (int i = 0; i < KEPT; ++i)
            if (r0 + i < r1 && token_row<STEP>(a, r0 + i, bad) < 0) kept[i] = 0;
#pragma unroll
    for (int i = 0; i < KEPT; ++i) {
        bad |= kept[i] < 0 || kept[i] > cap;
        kept[i] = clamp_len(kept[i], cap);
        mine += weight(units_of<D>(kept[i]));
    }
    for (int r = r0 + KEPT; r < r1; ++r) {
        const int n = token_row<STEP>(a, r, bad) < 0 ? 0 : a.lens[r];
        bad |= n < 0 || n > cap;
        mine += weight(units_of<D>(clamp_len(n, cap)));
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
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += sh[w];
        all += sh[w];
    }
    __syncthreads();
    Work k;
    k.total = all * rows;
    const long long most = (k.total + NW * MIN_SHARE - 1) / (NW * MIN_SHARE);
    k.grid = static_cast<int>(min(static_cast<long long>(a.grid), max(most, 1ll)));
    k.each = quotient(k.total, k.grid * NW);
    k.more = static_cast<int>(k.total - k.each * (k.grid * NW));
    const long long from = (before + x - mine) * rows, to = from + mine * rows;
    for (int w = 0; w < count; ++w) {
        if (first + w * step >= k.grid * NW) break;
        const long long s = k.start(first + w * step);
        if (s < from || s >= to) continue;
        long long at = from;
        int r = -1, un = 0, n = 0;
#pragma unroll
        for (int i = 0; i < KEPT; ++i) {
            if (r >= 0) continue;
            const long long next = at + static_cast<long long>(weight(units_of<D>(kept[i]))) * rows;
            if (s < next) r = r0 + i, n = kept[i];
            else at = next;
        }
        for (int i = r0 + KEPT; r < 0 && i < r1; ++i) {
            n = tokens_of<STEP>(a, i, cap);
            const long long next = at + static_cast<long long>(weight(units_of<D>(n))) * rows;
            if (s < next) r = i;
            else at = next;
        }
        if (r < 0) r = r1 - 1;
        un = units_of<D>(n);
        const int each_row = weight(un);
        const int row = static_cast<int>(
            min(quotient(s - at, max(each_row, 1)), static_cast<long long>(rows - 1)));
        sh[6 * w] = max(at + static_cast<long long>(row) * each_row, s - each_row);
        sh[6 * w + 1] = r;
        sh[6 * w + 2] = row;
        sh[6 * w + 3] = n;
    }
    return k;
}

template <int D>
__device__ __forceinline__ Row located(const long long* sh) {
    Row p;
    p.base = sh[0];
    p.r = static_cast<int>(sh[1]);
    p.row = static_cast<int>(sh[2]);
    p.n = static_cast<int>(sh[3]);
    p.units = units_of<D>(p.n);
    return p;
}

// the next row that has units (the caller knows that there is one)
template <int D, bool STEP>
__device__ __forceinline__ void next_row(const PagedAttnArgs& a, Row& p) {
    p.base += weight(p.units);
    if (++p.row < a.Hkv * a.head_tiles) return;
    p.row = 0;
    do {
        ++p.r;
        p.n = p.r < a.R ? tokens_of<STEP>(a, p.r, a.max_pages * a.page) : 1;
    } while (p.n == 0);
    p.r = min(p.r, a.R - 1);  // reached only if the lengths change meanwhile: stay within the table
    p.units = units_of<D>(p.n);
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

// where entry e's unnormalised output lies: a warp's part 0 in its own place, its part
// 1 in its ring
template <int D, int MT>
__device__ __forceinline__ float* part_o(uint8_t* smem, int e) {
    using C = Cfg<D, MT>;
    const int warp = e >> 1;
    return reinterpret_cast<float*>((e & 1) ? smem + warp * C::ST * C::STAGE
                                            : smem + C::OFF_O + warp * C::HEADS * D * 4);
}

// natural log of the softmax denominator from the base-2 maximum and sum
__device__ __forceinline__ float log_sum(float m, float l) {
    return ((m == -INFINITY ? 0.0f : m) + log2f(l)) * 0.6931471805599453f;
}

// zeros for the requests r, r + step, ... that have a row but no tokens
template <int D, bool STEP>
__device__ __forceinline__ void empty_rows(const PagedAttnArgs& a, int r, int step, int cap) {
    const int elems = a.H * D;
    for (; r < a.R; r += step) {
        if (clamp_len(a.lens[r], cap) > 0) continue;
        bool bad = false;
        const long long row = token_row<STEP>(a, r, bad);
        if (row < 0) continue;
        for (int i = threadIdx.x; i < elems / 8; i += NT)
            reinterpret_cast<uint4*>(a.o + row * elems)[i] = make_uint4(0, 0, 0, 0);
        if (a.lse)
            for (int h = threadIdx.x; h < a.H; h += NT) a.lse[row * a.H + h] = -INFINITY;
    }
}

// Four columns of a query head are an item of the CTA's join; a thread's items go side by
// side.
template <int D, int MT>
struct Joined {
    static constexpr int ITEMS = Cfg<D, MT>::HEADS * (D / 4) / NT;
    static constexpr int HSTEP = NT / (D / 4);
    static_assert(Cfg<D, MT>::HEADS * (D / 4) % NT == 0, "items of a thread");
    float top[ITEMS], sum[ITEMS];
    float4 acc[ITEMS];
    __device__ __forceinline__ int head(int k) const { return threadIdx.x / (D / 4) + k * HSTEP; }
    __device__ __forceinline__ int col() const { return 4 * (threadIdx.x % (D / 4)); }
};

__device__ __forceinline__ void add_scaled(float4& acc, float x, const float4& v) {
    acc.x += x * v.x, acc.y += x * v.y, acc.z += x * v.z, acc.w += x * v.w;
}
__device__ __forceinline__ float finite_ref(float m) { return m == -INFINITY ? 0.0f : m; }

// joins the entries `these` (bits) of the CTA's warps
template <int D, int MT>
__device__ __forceinline__ void join_entries(uint8_t* smem, uint32_t these, Joined<D, MT>& j) {
    using C = Cfg<D, MT>;
    const float* sm_m = reinterpret_cast<const float*>(smem + C::OFF_M) + j.head(0);
    const float* sm_l = reinterpret_cast<const float*>(smem + C::OFF_L) + j.head(0);
#pragma unroll
    for (int k = 0; k < j.ITEMS; ++k) {
        j.top[k] = -INFINITY, j.sum[k] = 0.0f;
        j.acc[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    for (uint32_t es = these; es; es &= es - 1) {
        const float* m = sm_m + (__ffs(es) - 1) * C::HEADS;
#pragma unroll
        for (int k = 0; k < j.ITEMS; ++k) j.top[k] = fmaxf(j.top[k], m[k * j.HSTEP]);
    }
    for (uint32_t es = these; es; es &= es - 1) {
        const int e = __ffs(es) - 1;
        const float* src = part_o<D, MT>(smem, e) + j.head(0) * D + j.col();
#pragma unroll
        for (int k = 0; k < j.ITEMS; ++k) {
            const float x = ex2_approx(sm_m[e * C::HEADS + k * j.HSTEP] - finite_ref(j.top[k]));
            j.sum[k] += x * sm_l[e * C::HEADS + k * j.HSTEP];
            add_scaled(j.acc[k], x, *reinterpret_cast<const float4*>(src + k * j.HSTEP * D));
        }
    }
}

// a finished query head's four columns (and its lse with the first)
template <int D>
__device__ __forceinline__ void store_head(const PagedAttnArgs& a, long long row, int col,
                                           const float4& acc, float top, float sum) {
    const float inv = 1.0f / sum;
    *reinterpret_cast<uint2*>(a.o + row * D + col) = make_uint2(
        pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (a.lse && col == 0) a.lse[row] = log_sum(top, sum);
}

__device__ __forceinline__ float peer_f(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float4 peer_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// The row of a cluster: every CTA joins its warps' parts, then each takes some of the
// heads' columns and reads the others' results from their shared memory.
template <int D, int MT, bool STEP>
__device__ __forceinline__ void join_cluster(const PagedAttnArgs& a, uint8_t* smem, const Row& p,
                                             uint32_t entries) {
    using C = Cfg<D, MT>;
    Joined<D, MT> j;
    join_entries<D, MT>(smem, entries, j);
    float* o = part_o<D, MT>(smem, 0);  // free: the parts lie in the rings
    float* stats = reinterpret_cast<float*>(smem + C::OFF_SH);  // maxima, sums
#pragma unroll
    for (int k = 0; k < j.ITEMS; ++k) {
        *reinterpret_cast<float4*>(o + j.head(k) * D + j.col()) = j.acc[k];
        if (j.col() == 0) stats[j.head(k)] = j.top[k], stats[C::HEADS + j.head(k)] = j.sum[k];
    }
    cluster_sync();
    const int hk = p.row / a.head_tiles, ht = p.row - hk * a.head_tiles;
    const int heads = min(a.tile_heads, a.group - ht * a.tile_heads);
    const long long q_row =
        static_cast<long long>(row_of<STEP>(a, p.r)) * a.H + hk * a.group + ht * a.tile_heads;
    const int n = a.whole_rows;
    for (int i = cluster_ctarank() * NT + threadIdx.x; i < heads * (D / 4); i += n * NT) {
        const int h = i / (D / 4), col = 4 * (i % (D / 4));
        const uint32_t so = smem_u32(o + h * D + col), sm = smem_u32(stats + h);
        float top = -INFINITY, sum = 0.0f;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int c = 0; c < n; ++c) top = fmaxf(top, peer_f(map_to_rank(sm, c)));
#pragma unroll 4
        for (int c = 0; c < n; ++c) {
            const float x = ex2_approx(peer_f(map_to_rank(sm, c)) - finite_ref(top));
            sum += x * peer_f(map_to_rank(sm + 4 * C::HEADS, c));
            add_scaled(acc, x, peer_f4(map_to_rank(so, c)));
        }
        store_head<D>(a, q_row + h, col, acc, top, sum);
    }
    cluster_sync();  // the others have read this CTA's shared memory
}

template <int D, int MT, bool STEP>
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
    const int cap = a.max_pages * a.page;

    if (threadIdx.x == 0) {
        *abort_flag = 0;
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
    }
    if (lane == 0)
        for (int s = 0; s < C::ST; ++s) mbar_init(bars + 8 * s, 1);
    fence_mbar_init();
    // the kernel before this one in the stream may still run (an append, say: its CTAs let this
    // grid in early): nothing in memory is touched before it has ended. Then the
    // joining kernel's CTAs may settle on the SMs and read the lengths; they wait for this
    // grid's end in turn
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");

    const int cta = blockIdx.x, rows = a.Hkv * a.head_tiles;
    long long g0, g1;  // this warp's share: units g0 .. g1 - 1
    Row p;
    if (a.whole_rows) {
        // a row per CTA or cluster, an equal part of it per warp
        const int row = cta / a.whole_rows, piece = (cta - row * a.whole_rows) * NW + warp;
        p.base = 0;
        p.r = row / rows;
        p.row = row - p.r * rows;
        bool bad = false;
        const int n = token_row<STEP>(a, p.r, bad) < 0 ? 0 : a.lens[p.r];
        p.n = clamp_len(n, cap);
        p.units = units_of<D>(p.n);
        bad |= n != p.n;
        if (p.row == 0 && threadIdx.x == 0 && bad && a.status)
            atomicOr(a.status, VELOX_STATUS_BAD_INDEX);
        const int pieces = a.whole_rows * NW;
        g0 = static_cast<long long>(p.units) * piece / pieces;
        g1 = static_cast<long long>(p.units) * (piece + 1) / pieces;
        __syncthreads();  // barriers initialised
        if (p.n == 0) {
            if (p.row == 0 && piece < NW) empty_rows<D, STEP>(a, p.r, a.R, cap);
            if (a.whole_rows > 1) {
                // in step with the cluster to its end, should others have seen a length
                if (lane < 2) reinterpret_cast<int*>(smem + C::OFF_ENT)[8 * warp + 4 * lane] = -1;
                __syncthreads();
                cluster_sync();
                cluster_sync();
            }
            return;
        }
    } else {
        const Work work = locate<D, STEP, NT>(a, cta * NW, NW, 1, sh, cta == 0);
        __syncthreads();  // rows found, barriers initialised
        if (cta >= work.grid || work.total == 0) {
            empty_rows<D, STEP>(a, cta, gridDim.x, cap);
            return;
        }
        g0 = work.start(cta * NW + warp), g1 = work.start(cta * NW + warp + 1);
        p = located<D>(sh + 6 * warp);
    }

    // ---- loads, ahead of the products and across rows. f: the row of the next unit to
    // fetch, fu .. fend - 1 what is left of it in the share. Lane i keeps the page id of
    // the row's box ids_at + i
    constexpr int SUB = C::SUB, UNIT = C::UNIT;
    Row f = p;
    int fu = 0, fend = 0, ids_at = 0, ids = 0;
    // units are left to fetch (test hook: a warp that fetches nothing waits in vain)
    bool more = g0 < g1 && !(a.skip_warps >> warp & 1);
    const auto look_up = [&]() {
        ids_at = fu * SUB;
        const int box = ids_at + lane;
        if (box < fend * SUB && box * BOX < f.n)
            ids = a.table[static_cast<long long>(f.r) * a.max_pages + ((box * BOX) >> a.page_shift)];
    };
    if (more) {
        fu = static_cast<int>(g0 - f.base);
        fend = static_cast<int>(min(g1 - f.base, static_cast<long long>(f.units)));
    }
    const auto settle = [&]() {  // fu to a unit that is there, its page ids to lanes
        while (more && fu >= fend) {
            if (f.base + weight(f.units) >= g1) {
                more = false;
            } else {
                next_row<D, STEP>(a, f);
                fu = 0;
                fend = static_cast<int>(min(g1 - f.base, static_cast<long long>(f.units)));
                ids_at = -32;
            }
        }
        if (more && (fu + 1) * SUB - ids_at > 32) look_up();
    };
    ids_at = fu * SUB - 32;
    settle();
    const auto fetch = [&](int slot) {
        int found[SUB];
#pragma unroll
        for (int i = 0; i < SUB; ++i) {
            found[i] = __shfl_sync(~0u, ids, fu * SUB + i - ids_at);
            // a last unit may end in its first box: the second then is any page that is there
            if (i > 0 && (fu * SUB + i) * BOX >= f.n) found[i] = found[0];
        }
        if (lane == 0) {
            const uint32_t bar = bars + 8 * slot, dst = ring + slot * C::STAGE;
            mbar_arrive_expect_tx(bar, C::STAGE);
            int y[SUB];
#pragma unroll
            for (int i = 0; i < SUB; ++i) {
                int id = found[i];
                if (id < 0 || id >= a.num_pages) {
                    if (a.status) atomicOr(a.status, VELOX_STATUS_BAD_INDEX);
                    id = 0;
                }
                y[i] = (id * a.Hkv + f.row / a.head_tiles) * a.page +
                       (((fu * SUB + i) * BOX) & (a.page - 1));
            }
            // D = 128: the two column halves of a box; D = 64: two boxes
#pragma unroll
            for (int i = 0; i < 2; ++i)
                tma_load_2d(dst + i * C::HALF, &tmK, bar, SUB == 1 ? 64 * i : 0, y[SUB == 1 ? 0 : i]);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                tma_load_2d(dst + C::TILE + i * C::HALF, &tmV, bar, SUB == 1 ? 64 * i : 0,
                            y[SUB == 1 ? 0 : i]);
        }
        ++fu;
        settle();
    };
    int ahead = 0;  // units fetched and not yet used
    for (int s = 0; s < a.stages; ++s)
        if (more) {
            fetch(s);
            ++ahead;
        }

    if (!a.whole_rows) empty_rows<D, STEP>(a, cta, gridDim.x, cap);  // while the loads are on their way

    const int g = lane >> 2, t = lane & 3;
    int* ent = reinterpret_cast<int*>(smem + C::OFF_ENT) + 8 * warp;  // this warp's two parts
    if (lane < 2) ent[4 * lane] = -1;  // none yet
    const bool clustered = a.whole_rows > 1;
    int slot = 0;
    uint32_t parity = 0;
    bool ok = true;
    while (g0 < g1) {
        // units of this row in the share
        const int u0 = static_cast<int>(max(g0 - p.base, 0ll));
        const int u1 = static_cast<int>(min(g1 - p.base, static_cast<long long>(p.units)));
        if (u0 < u1) {
            const int hk = p.row / a.head_tiles, ht = p.row - hk * a.head_tiles;
            const int head0 = hk * a.group + ht * a.tile_heads;
            const int heads = min(a.tile_heads, a.group - ht * a.tile_heads);
            const long long q_row = static_cast<long long>(row_of<STEP>(a, p.r)) * a.H + head0;

            float o[MT][D / 8][4];
            float m[MT], l[MT];
            uint32_t q[MT][D / 16][2];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                m[i] = -INFINITY, l[i] = 0.0f;
#pragma unroll
                for (int j = 0; j < D / 8; ++j)
                    o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.0f;
                const bool have = 8 * i + g < heads;
                const uint32_t* src =
                    reinterpret_cast<const uint32_t*>(a.q + (q_row + (have ? 8 * i + g : 0)) * D) + t;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    q[i][k][0] = have ? src[8 * k] : 0u;
                    q[i][k][1] = have ? src[8 * k + 4] : 0u;
                }
            }
            for (int u = u0; u < u1; ++u) {
                ok = mbar_wait(bars + 8 * slot, parity, abort_flag, a.wait_ns);
                ok = __all_sync(~0u, ok);
                if (!ok) break;
                const uint32_t kt = ring + slot * C::STAGE, vt = kt + C::TILE;
                const int valid = p.n - u * UNIT;  // tokens left
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
                // S: two key groups of 8 per box, at d = 128 each in two chains over d
                constexpr int KG = 2 * SUB, CH = SUB == 1 ? 2 : 1;
                float s[CH][KG][4];
#pragma unroll
                for (int i = 0; i < CH; ++i)
#pragma unroll
                    for (int j = 0; j < KG; ++j) s[i][j][0] = s[i][j][1] = s[i][j][2] = s[i][j][3] = 0.0f;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t a1 = MT == 2 ? q[MT - 1][k][0] : 0u;
                    const uint32_t a3 = MT == 2 ? q[MT - 1][k][1] : 0u;
#pragma unroll
                    for (int x = 0; x < SUB; ++x) {
                        uint32_t b[4];  // keys 0-7 of the box: d lo, d hi; keys 8-15: d lo, d hi
                        ldsm4(kt + tile_at<D, MT>(BOX * x + (lane & 7) + ((lane >> 4) << 3),
                                                  2 * k + ((lane >> 3) & 1)),
                              b);
                        mma16816(s[k % CH][2 * x], q[0][k][0], a1, q[0][k][1], a3, b[0], b[1]);
                        mma16816(s[k % CH][2 * x + 1], q[0][k][0], a1, q[0][k][1], a3, b[2], b[3]);
                    }
                }
                uint32_t hi[MT][KG], lo[MT][KG];
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    float x[2 * KG];  // keys 8 j + 2t, 8 j + 2t + 1 of head 8 i + g
                    float top = -INFINITY;
#pragma unroll
                    for (int j = 0; j < 2 * KG; ++j) {
                        x[j] = s[0][j >> 1][2 * i + (j & 1)];
                        if (CH == 2) x[j] += s[CH - 1][j >> 1][2 * i + (j & 1)];
                        x[j] *= a.scale_log2;
                        if (8 * (j >> 1) + 2 * t + (j & 1) >= valid) x[j] = -INFINITY;
                        top = fmaxf(top, x[j]);
                    }
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
                    const float ref = finite_ref(m[i]);
#pragma unroll
                    for (int j = 0; j < KG; ++j) {
                        const float p0 = ex2_approx(x[2 * j] - ref), p1 = ex2_approx(x[2 * j + 1] - ref);
                        l[i] += p0 + p1;
                        hi[i][j] = pack_bf16x2(p0, p1);
                        lo[i][j] = pack_bf16x2(p0 - bf16_lo(hi[i][j]), p1 - bf16_hi(hi[i][j]));
                    }
                }
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
#pragma unroll
                    for (int x = 0; x < SUB; ++x) {
                        uint32_t b[4];  // d 16 j .. +7: keys lo, keys hi; the next 8: keys lo, keys hi
                        ldsm4_t(vt + tile_at<D, MT>(BOX * x + (lane & 7) + (((lane >> 3) & 1) << 3),
                                                    2 * j + (lane >> 4)),
                                b);
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            const uint32_t h0 = hi[i][2 * x], h1 = hi[i][2 * x + 1];
                            const uint32_t l0 = lo[i][2 * x], l1 = lo[i][2 * x + 1];
                            mma16816(o[i][2 * j], h0, l0, h1, l1, b[0], b[1]);
                            mma16816(o[i][2 * j + 1], h0, l0, h1, l1, b[2], b[3]);
                        }
                    }
                }
                __syncwarp();  // every lane has read the slot
                --ahead;
                if (more) {
                    fetch(slot);
                    ++ahead;
                }
                if (++slot == a.stages) slot = 0, parity ^= 1;
            }
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                l[i] += __shfl_xor_sync(~0u, l[i], 1);
                l[i] += __shfl_xor_sync(~0u, l[i], 2);
#pragma unroll
                for (int j = 0; j < D / 8; ++j) {
                    if (isfinite(o[i][j][2])) o[i][j][0] += o[i][j][2];
                    if (isfinite(o[i][j][3])) o[i][j][1] += o[i][j][3];
                }
            }
            const bool begins = u0 == 0, ends = u1 == p.units;
            if (begins && ends && !clustered) {
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    if (8 * i + g < heads) {
                        const float inv = 1.0f / l[i];
                        uint32_t* dst =
                            reinterpret_cast<uint32_t*>(a.o + (q_row + 8 * i + g) * D) + t;
#pragma unroll
                        for (int j = 0; j < D / 8; ++j)
                            dst[4 * j] = pack_bf16x2(o[i][j][0] * inv, o[i][j][1] * inv);
                        if (a.lse && t == 0) a.lse[q_row + 8 * i + g] = log_sum(m[i], l[i]);
                    }
            } else {
                // part 0: the end of a row that another warp began; part 1: a row that
                // goes on in the next warp (or any part of a cluster's row). Part 1 is this
                // warp's last row, so its ring has no load in flight
                const int k = ends && !clustered ? 0 : 1, e = 2 * warp + k;
                float* sm_o = part_o<D, MT>(smem, e);
                float* sm_m = reinterpret_cast<float*>(smem + C::OFF_M) + e * C::HEADS;
                float* sm_l = reinterpret_cast<float*>(smem + C::OFF_L) + e * C::HEADS;
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    if (t == 0) sm_m[8 * i + g] = m[i], sm_l[8 * i + g] = l[i];
                    if (8 * i + g < heads)
#pragma unroll
                        for (int j = 0; j < D / 8; ++j)
                            *reinterpret_cast<float2*>(sm_o + (8 * i + g) * D + 8 * j + 2 * t) =
                                make_float2(o[i][j][0], o[i][j][1]);
                }
                if (lane == 0) {
                    int* mine = ent + 4 * k;
                    mine[1] = p.r;
                    mine[2] = p.row;
                    mine[3] = begins;
                    mine[0] = 1;
                }
            }
        }
        if (p.base + weight(p.units) >= g1) break;
        next_row<D, STEP>(a, p);
    }
    // a wait that ran out: what is still in flight lands before the CTA leaves
    if (!ok || ahead > 0) {
        if (!ok && lane == 0 && a.status) atomicOr(a.status, VELOX_STATUS_TIMEOUT);
        volatile int never = 0;
        for (; ahead > 0; --ahead) {
            if (!mbar_wait(bars + 8 * slot, parity, &never, WAIT_LIMIT_NS)) break;
            if (++slot == a.stages) slot = 0, parity ^= 1;
        }
    }

    // ---- rows that several warps worked on. In the order of the entries, a row's parts
    // follow one another: parts 1 (it goes on), then a part 0 (it ends) if it ends
    // in this CTA
    __syncthreads();
    const int* ents = reinterpret_cast<const int*>(smem + C::OFF_ENT);
    uint32_t left = 0;  // bit e: an entry
#pragma unroll
    for (int e = 0; e < 2 * NW; ++e) left |= (ents[4 * e] >= 0 ? 1u : 0u) << e;
    if (clustered) {
        join_cluster<D, MT, STEP>(a, smem, p, left);
        return;
    }
    while (left) {
        const int e0 = __ffs(left) - 1;
        const uint32_t enders = left & 0x55555555u;
        const bool begins = ents[4 * e0 + 3] != 0, ends = enders != 0;
        const uint32_t these = ends ? left & ((2u << (__ffs(enders) - 1)) - 1) : left;
        left &= ~these;
        const int r = ents[4 * e0 + 1], row = ents[4 * e0 + 2];
        const int hk = row / a.head_tiles, ht = row - hk * a.head_tiles;
        const int heads = min(a.tile_heads, a.group - ht * a.tile_heads);
        const long long q_row =
            static_cast<long long>(row_of<STEP>(a, r)) * a.H + hk * a.group + ht * a.tile_heads;
        float* part = a.part + static_cast<long long>(2 * cta + (begins ? 1 : 0)) * C::PART;
        Joined<D, MT> j;
        join_entries<D, MT>(smem, these, j);
#pragma unroll
        for (int k = 0; k < j.ITEMS; ++k) {
            const int h = j.head(k), col = j.col();
            if (h >= heads) break;
            if (begins && ends) {
                store_head<D>(a, q_row + h, col, j.acc[k], j.top[k], j.sum[k]);
            } else if (!a.whole_rows) {
                // (a CTA's own row lacks entries only after a wait that ran out, and then
                // there may be no workspace)
                *reinterpret_cast<float4*>(part + h * D + col) = j.acc[k];
                if (col == 0) {
                    part[C::HEADS * D + h] = j.top[k];
                    part[C::HEADS * D + C::HEADS + h] = j.sum[k];
                }
            }
        }
    }
}

// Joins the parts of the rows that more than one CTA worked on. CTA c stands for share
// c, and the n shares of a row divide its query heads: heads i, i + n, ... fall to
// the i-th. Where there are more heads than shares (few parts each), a warp joins a
// head alone; where there are more shares (many parts), the CTA's warps take parts
// of one head in turn and meet in shared memory. The order of the sums is fixed.
template <int D, int MT, bool STEP>
__global__ void __launch_bounds__(JT)
    paged_join_kernel(const __grid_constant__ PagedAttnArgs a) {
    using C = Cfg<D, MT>;
    constexpr int LANES = D / 4, SUB = 32 / LANES;  // lanes of a part, parts at a time
    constexpr int AT_ONCE = 4;                      // parts of a lane loaded before their weights
    __shared__ long long sh[6 * JW];
    __shared__ float red_m[JW], red_l[JW];
    __shared__ float4 red_o[JW][LANES];
    const int c = blockIdx.x;
    const Work work = locate<D, STEP, JT>(a, c * NW, 2, NW, sh, false);
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the row that share c goes on with, and the one it begins and leaves. All of this
    // comes from the lengths, before the parts are there
    int first[2] = {}, n[2] = {}, heads[2] = {};
    long long q_row[2] = {};
    if (c < work.grid && work.total > 0) {
        const long long s0 = work.start(c * NW), s1 = work.start((c + 1) * NW);
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            if (side == 1 && c + 1 >= work.grid) break;
            const Row p = located<D>(sh + 6 * side);
            const long long end = p.base + p.units;
            if (side == 0 ? (s0 <= p.base || s0 >= end)
                          : (p.base < s0 || s1 <= p.base || s1 >= end))
                continue;
            first[side] = work.cta_of(p.base);
            n[side] = work.cta_of(end - 1) - first[side] + 1;
            const int hk = p.row / a.head_tiles, ht = p.row - hk * a.head_tiles;
            heads[side] = min(a.tile_heads, a.group - ht * a.tile_heads);
            q_row[side] =
                static_cast<long long>(row_of<STEP>(a, p.r)) * a.H + hk * a.group + ht * a.tile_heads;
        }
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");

    for (int side = 0; side < 2; ++side) {
        const int n_parts = n[side], begin = first[side], n_heads = heads[side];
        const bool team = n_parts >= n_heads;  // the whole CTA on one head
        const int step = team ? JW : 1;
        for (int hh = c - begin + (team ? 0 : n_parts * warp); hh < n_heads;
             hh += team ? n_parts : n_parts * JW) {
            // this warp's parts: i0, i0 + step, ...; lane j looks after the j-th, the
            // j + 32-th, ... (a team's warp has at most MAX_GRID / JW, a lone one 15)
            const int i0 = team ? warp : 0;
            const int mine = i0 < n_parts ? (n_parts - 1 - i0) / step + 1 : 0;
            // part 1 of the share in which the row begins, part 0 of the others
            const auto part_at = [&](int j) {
                const int i = i0 + j * step;
                return a.part + static_cast<long long>(2 * (begin + i) + (i == 0 ? 1 : 0)) * C::PART;
            };
            const int sub = lane / LANES, col = 4 * (lane % LANES);
            float4 v[AT_ONCE];
#pragma unroll
            for (int k = 0; k < AT_ONCE; ++k)
                if (k * SUB + sub < mine)
                    v[k] = *reinterpret_cast<const float4*>(part_at(k * SUB + sub) + hh * D + col);
            float m[PPL], l[PPL], w[PPL], top = -INFINITY;
#pragma unroll
            for (int k = 0; k < PPL; ++k) {
                m[k] = -INFINITY, l[k] = 0.0f;
                if (lane + 32 * k < mine) {
                    const float* part = part_at(lane + 32 * k);
                    m[k] = part[C::HEADS * D + hh];
                    l[k] = part[C::HEADS * D + C::HEADS + hh];
                }
                top = fmaxf(top, m[k]);
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
            const float ref = top == -INFINITY ? 0.0f : top;
            float sum = 0.0f;
#pragma unroll
            for (int k = 0; k < PPL; ++k) {
                w[k] = ex2_approx(m[k] - ref);
                sum += w[k] * l[k];
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int j = 0; j < mine; j += AT_ONCE * SUB) {
#pragma unroll
                for (int k = 0; k < AT_ONCE; ++k) {
                    const int at = j + k * SUB + sub;
                    float mine_w = w[0];  // at >> 5 is the same in all lanes
#pragma unroll
                    for (int i = 1; i < PPL; ++i) mine_w = (at >> 5) == i ? w[i] : mine_w;
                    const float x = __shfl_sync(~0u, mine_w, at & 31);
                    if (at < mine)
                        acc.x += x * v[k].x, acc.y += x * v[k].y, acc.z += x * v[k].z,
                            acc.w += x * v[k].w;
                }
#pragma unroll
                for (int k = 0; k < AT_ONCE; ++k) {
                    const int at = j + (AT_ONCE + k) * SUB + sub;
                    if (at < mine)
                        v[k] = *reinterpret_cast<const float4*>(part_at(at) + hh * D + col);
                }
            }
            if (SUB == 2) {
                acc.x += __shfl_xor_sync(~0u, acc.x, 16), acc.y += __shfl_xor_sync(~0u, acc.y, 16);
                acc.z += __shfl_xor_sync(~0u, acc.z, 16), acc.w += __shfl_xor_sync(~0u, acc.w, 16);
            }
            if (team) {
                if (lane == 0) red_m[warp] = top, red_l[warp] = sum;
                if (sub == 0) red_o[warp][lane] = acc;
                __syncthreads();
                if (warp == 0) {
                    top = red_m[0];
#pragma unroll
                    for (int k = 1; k < JW; ++k) top = fmaxf(top, red_m[k]);
                    const float all = top == -INFINITY ? 0.0f : top;
                    sum = 0.0f;
                    acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                    for (int k = 0; k < JW; ++k) {
                        const float x = ex2_approx(red_m[k] - all);
                        const float4 v = red_o[k][lane % LANES];
                        sum += x * red_l[k];
                        acc.x += x * v.x, acc.y += x * v.y, acc.z += x * v.z, acc.w += x * v.w;
                    }
                }
                __syncthreads();
            }
            if ((!team || warp == 0) && sub == 0) {
                const float inv = 1.0f / sum;
                *reinterpret_cast<uint2*>(a.o + (q_row[side] + hh) * D + col) = make_uint2(
                    pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
                if (a.lse && lane == 0) a.lse[q_row[side] + hh] = log_sum(top, sum);
            }
        }
    }
}

// CTAs per row where rows are not dealt out by length, else 0: those of a short history
// (paged_attn_whole); a cluster for a single request, whose rows are all of one length, where
// clusters of 16, 10 or 8 (sizes that the GPU holds at once, with two CTAs per SM) make up a
// grid that fills it. 24 key heads, one launch against two: 4096 tokens (in L2) 12.6 and 15.5
// us, 32,768 tokens 64.8 and 67.5, 225,793 tokens 389 and 403 (in a steady loop under the
// power cap 402 and 406; clusters of 8: 13.0, 65.3, 412, steady 447; of 11, which do not fit:
// 21.5, 100, 625). 8 key heads (128 CTAs, not taken): 10.4 and 12.1 us at 4096 tokens, 203 and
// 141 at 225,793.
// places(n): the device can place a cluster of n CTAs, more than the 8 that any can.
template <typename F>
int ctas_per_row(const PagedAttnArgs& a, long long rows, F places) {
    if (a.whole_rows || a.R > 1) return a.whole_rows;
    for (const int n : {16, 10, 8})
        if (rows * n <= 256 && rows * n >= 160 && n <= a.most_cluster && (n <= 8 || places(n)))
            return n;
    return 0;
}

// Whether the current device can place a cluster of n of the kernel's CTAs: a part of a GPU may
// be too small for it. `known` keeps the answer (0: not asked yet, 1: no, 2: yes).
template <typename K>
bool can_place(K kern, int n, size_t smem, std::atomic<int>& known) {
    int answer = known.load(std::memory_order_relaxed);
    if (answer == 0) {
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = n;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(n);
        cfg.blockDim = dim3(NT);
        cfg.dynamicSmemBytes = smem;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        int clusters = 0;
        const bool asked =
            cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
            cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg) == cudaSuccess;
        if (!asked) cudaGetLastError();  // the refusal is the answer, not the call's error
        answer = asked && clusters > 0 ? 2 : 1;
        known.store(answer, std::memory_order_relaxed);
    }
    return answer == 2;
}

template <int D, int MT, bool STEP>
int launch(const void* k_pages, const void* v_pages, PagedAttnArgs a, cudaStream_t st) {
    using C = Cfg<D, MT>;
    static_assert(C::SMEM + 1024 <= 233472 / 2, "shared memory of two CTAs");
    static_assert(C::HALF % 1024 == 0, "swizzle atoms");
    CUtensorMap tk, tv;
    const uint64_t pool = static_cast<uint64_t>(a.num_pages) * a.Hkv * a.page;
    if (!make_tmap(&tk, k_pages, pool, D, BOX) || !make_tmap(&tv, v_pages, pool, D, BOX))
        return VELOX_ECUDA;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return VELOX_ECUDA;
    // a ragged batch of 64 requests: 78.4 us, 87.9 with one CTA per SM, 79.6 with two
    const int resident = std::min(7 * sms / 4, MAX_GRID);
    const long long rows = static_cast<long long>(a.R) * a.Hkv * a.head_tiles;
    const long long units = static_cast<long long>(a.max_pages) * a.page / C::UNIT + 1;
    auto kern = paged_attn_kernel<D, MT, STEP>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) !=
        cudaSuccess)
        return VELOX_ECUDA;
    constexpr int DEVICES = 64;  // beyond these no cluster of more than 8 is taken
    static std::atomic<int> known[DEVICES][2];
    a.whole_rows = ctas_per_row(a, rows, [&](int n) {
        return dev < DEVICES && can_place(kern, n, C::SMEM, known[dev][n == 16]);
    });
    // no more CTAs than the longest histories could keep busy
    a.grid = static_cast<int>(
        a.whole_rows ? rows * a.whole_rows
                     : std::min<long long>(resident, (rows * (units + ROW_COST) + NW * MIN_SHARE - 1) /
                                                         (NW * MIN_SHARE)));
    // units in flight: as many as come nearest to IN_FLIGHT bytes on the whole GPU
    const double per_stage = static_cast<double>(a.grid) * NW * C::STAGE;
    a.stages = std::max(2, std::min(C::ST, static_cast<int>(IN_FLIGHT / per_stage + 0.5)));
    if (a.whole_rows > 8 &&
        cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
        return VELOX_ECUDA;
    // the launch overlaps the end of the kernel before it: append and attention of a layer take
    // 8.7 us instead of 9.4 at 300 tokens of 24 heads, 26.7 instead of 27.6 at 9000
    cudaLaunchAttribute at[2];
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(a.grid);
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (a.whole_rows > 1) {
        at[1].id = cudaLaunchAttributeClusterDimension;
        at[1].val.clusterDim.x = a.whole_rows;
        at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    if (cudaLaunchKernelEx(&cfg, kern, tk, tv, a) != cudaSuccess) return VELOX_ECUDA;
    if (a.whole_rows || a.grid == 1) return VELOX_OK;  // no row is shared between shares
    cfg.blockDim = dim3(JT);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, paged_join_kernel<D, MT, STEP>, a) == cudaSuccess ? VELOX_OK
                                                                               : VELOX_ECUDA;
}

}  // namespace

int paged_attn_whole(int R, int H, int Hkv, int page, int max_pages) {
    const long long rows = static_cast<long long>(R) * Hkv * ((H / Hkv + 15) / 16);
    const long long tokens = static_cast<long long>(max_pages) * page;
    int n = 8;
    while (n > 0 && rows * n > WHOLE_CTAS) n /= 2;
    if (tokens > static_cast<long long>(WHOLE_TOKENS) * n) return 0;
    while (n > 1 && tokens < NW / 2 * BOX * n) n /= 2;  // a box for every other warp
    return n;
}

size_t paged_attn_ws_bytes(int R, int H, int Hkv, int d) {
    const int mt = H / Hkv > 8 ? 2 : 1;
    return static_cast<size_t>(2 * MAX_GRID) * 8 * mt * (d + 2) * sizeof(float);
}

int paged_attn_launch(const void* k_pages, const void* v_pages, const PagedAttnArgs& args, int d,
                      cudaStream_t st) {
    PagedAttnArgs a = args;
    a.group = a.H / a.Hkv;
    a.head_tiles = (a.group + 15) / 16;
    a.whole_rows = paged_attn_whole(a.R, a.H, a.Hkv, a.page, a.max_pages);
    a.tile_heads = (a.group + a.head_tiles - 1) / a.head_tiles;
    const bool wide = a.group > 8, step = a.cu != nullptr;
    const auto run = [&](auto kernel) { return kernel(k_pages, v_pages, a, st); };
    if (d == 128)
        return step ? run(wide ? launch<128, 2, true> : launch<128, 1, true>)
                    : run(wide ? launch<128, 2, false> : launch<128, 1, false>);
    return step ? run(wide ? launch<64, 2, true> : launch<64, 1, true>)
                : run(wide ? launch<64, 2, false> : launch<64, 1, false>);
}

}  // namespace velox
