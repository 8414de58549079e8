// Block tables and slot maps of a paged KV cache, built on the GPU from the
// requests' lengths, and pages given back.
//
// Per request r: need_r = ceil((lens+add)/page) - ceil(lens/page) pages. Their
// exclusive prefix sum P_r places them on the stack of free pages (request r's
// i-th new page is free_list[free_count - 1 - P_r - i]), that of `add` places
// its tokens. Integer work on a few kilobytes: what bounds it is latency, the
// launch and the chain read lengths -> scan -> read pages -> write slots. So one
// launch does all of it: the CTAs of one cluster scan the same lengths each
// (8192 requests are 64 KB), keep the prefix sums in shared memory, and share the
// pages and the tokens. Cluster barriers stand between reading the lengths and
// writing them (outputs may be inputs) and between entering pages and
// reading them for the slots.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "ptx.cuh"
#include "velox_internal.cuh"

namespace velox {

namespace {

constexpr int PT = 1024;      // threads per CTA
constexpr int PWARPS = PT / 32;

// exclusive prefix over the CTA of two 64-bit values, and their totals
__device__ __forceinline__ void scan2(long long& a, long long& b, long long& ta, long long& tb,
                                      long long* sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long x = a, y = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(~0u, x, o), v = __shfl_up_sync(~0u, y, o);
        if (lane >= o) x += u, y += v;
    }
    if (lane == 31) sh[warp] = x, sh[PWARPS + warp] = y;
    __syncthreads();
    if (warp == 0) {
        long long p = sh[lane], q = sh[PWARPS + lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(~0u, p, o), v = __shfl_up_sync(~0u, q, o);
            if (lane >= o) p += u, q += v;
        }
        sh[lane] = p, sh[PWARPS + lane] = q;
    }
    __syncthreads();
    ta = sh[PWARPS - 1], tb = sh[2 * PWARPS - 1];
    a = x - a + (warp ? sh[warp - 1] : 0);
    b = y - b + (warp ? sh[PWARPS + warp - 1] : 0);
}

// largest r in [0, R) with p[r] <= x, for p ascending with p[0] = 0
__device__ __forceinline__ int owner(const int* p, int R, int x) {
    int lo = 0, hi = R;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ int pages_of(int tokens, int page) {
    return static_cast<int>((static_cast<long long>(tokens) + page - 1) / page);
}

__device__ __forceinline__ void flag(int32_t* status, int bit) {
    if (status) atomicOr(status, bit);
}

// shared memory: int tok[R + 1] (plan), pg[R + 1], old[R + 1]
__global__ void __launch_bounds__(PT, 1) paged_plan_kernel(const __grid_constant__ PlanArgs a) {
    extern __shared__ int sm[];
    __shared__ long long sh[2 * PWARPS];
    __shared__ int bad_any;
    int* tok = sm;
    int* pg = tok + a.R + 1;
    int* old = pg + a.R + 1;
    const int rank = cluster_ctarank(), ctas = gridDim.x;
    const long long cap = static_cast<long long>(a.max_pages) * a.page;
    const int per = (a.R + PT - 1) / PT;
    const int r0 = min(a.R, static_cast<int>(threadIdx.x) * per), r1 = min(a.R, r0 + per);

    if (threadIdx.x == 0) bad_any = 0;
    __syncthreads();
    const int fc = *a.free_count;
    // bit 0: a length that cannot be, bit 1: a request beyond its table row
    int bad = (fc < 0 || fc > a.num_pages) ? 1 : 0;
    long long nt = 0, np = 0;
    for (int r = r0; r < r1; ++r) {
        const int n = a.lens[r], m = a.add[r];
        if (n < 0 || n > cap || m < 0) {
            bad |= 1;
            continue;
        }
        if (static_cast<long long>(n) + m > cap) {
            bad |= 2;
            continue;
        }
        nt += m;
        np += pages_of(n + m, a.page) - pages_of(n, a.page);
    }
    if (bad) atomicOr(&bad_any, bad);
    long long t0 = nt, p0 = np, tt, tp;
    scan2(t0, p0, tt, tp, sh);  // its barriers also order bad_any
    const int worst = bad_any;
    const bool ok = worst == 0 && tp <= fc && tt <= a.n_cap;
    int tokens = 0, new_pages = 0;
    if (ok) {
        tokens = static_cast<int>(tt);
        new_pages = static_cast<int>(tp);
        int t = static_cast<int>(t0), p = static_cast<int>(p0);
        for (int r = r0; r < r1; ++r) {
            const int n = a.lens[r], m = a.add[r];
            const int o = pages_of(n, a.page);
            tok[r] = t;
            pg[r] = p;
            old[r] = n;
            t += m;
            p += pages_of(n + m, a.page) - o;
        }
        if (threadIdx.x == 0) tok[a.R] = tokens, pg[a.R] = new_pages;
    }
    // every CTA has read the lengths and the count: they may be overwritten
    cluster_sync();

    const int gtid = rank * PT + threadIdx.x, all = ctas * PT;
    if (rank == 0) {
        for (int r = threadIdx.x; r < a.R; r += PT) {
            a.cu[r] = ok ? tok[r] : 0;
            if (ok) a.lens_out[r] = old[r] + tok[r + 1] - tok[r];
            else if (a.lens_out != a.lens) a.lens_out[r] = a.lens[r];
        }
        if (threadIdx.x == 0) {
            a.cu[a.R] = tokens;
            *a.free_count_out = fc - new_pages;
            if (!ok)
                flag(a.status, (worst & 1) ? VELOX_STATUS_BAD_INDEX : VELOX_STATUS_NO_SPACE);
        }
    }
    for (int p = gtid; p < new_pages; p += all) {
        const int r = owner(pg, a.R, p);
        const int col = pages_of(old[r], a.page) + p - pg[r];
        a.table[static_cast<long long>(r) * a.max_pages + col] = a.free_list[fc - 1 - p];
    }
    cluster_sync();  // pages entered by any CTA of the cluster are visible

    bool stray = false;
    for (int t = gtid; t < a.n_cap; t += all) {
        int slot = -1, pos = -1, r = -1;
        if (t < tokens) {
            r = owner(tok, a.R, t);
            pos = old[r] + t - tok[r];
            const int id = a.table[static_cast<long long>(r) * a.max_pages + pos / a.page];
            if (id >= 0 && id < a.num_pages) slot = id * a.page + pos % a.page;
            else stray = true;
        }
        a.slots[t] = slot;
        if (a.pos) a.pos[t] = pos;
        if (a.req) a.req[t] = r;
    }
    if (stray) flag(a.status, VELOX_STATUS_BAD_INDEX);
}

// shared memory: int pg[R + 1]
__global__ void __launch_bounds__(PT, 1) paged_release_kernel(const __grid_constant__ PlanArgs a) {
    extern __shared__ int sm[];
    __shared__ long long sh[2 * PWARPS];
    __shared__ int bad_any;
    int* pg = sm;
    const int rank = cluster_ctarank(), ctas = gridDim.x;
    const long long cap = static_cast<long long>(a.max_pages) * a.page;
    const int per = (a.R + PT - 1) / PT;
    const int r0 = min(a.R, static_cast<int>(threadIdx.x) * per), r1 = min(a.R, r0 + per);

    if (threadIdx.x == 0) bad_any = 0;
    __syncthreads();
    const int fc = *a.free_count;
    int bad = (fc < 0 || fc > a.num_pages) ? 1 : 0;
    long long np = 0, zero = 0;
    for (int r = r0; r < r1; ++r) {
        const int n = a.lens[r];
        if (n < 0 || n > cap) bad = 1;
        else if (a.add[r] != 0) np += pages_of(n, a.page);
    }
    if (bad) atomicOr(&bad_any, bad);
    long long p0 = np, tp, tz;
    scan2(p0, zero, tp, tz, sh);
    const bool ok = bad_any == 0 && fc + tp <= a.num_pages;
    const int back = ok ? static_cast<int>(tp) : 0;
    if (ok) {
        int p = static_cast<int>(p0);
        for (int r = r0; r < r1; ++r) {
            pg[r] = p;
            if (a.add[r] != 0) p += pages_of(a.lens[r], a.page);
        }
    }
    cluster_sync();  // lengths and count read by every CTA

    if (rank == 0) {
        for (int r = threadIdx.x; r < a.R; r += PT)
            a.lens_out[r] = (ok && a.add[r] != 0) ? 0 : a.lens[r];
        if (threadIdx.x == 0) {
            *a.free_count_out = fc + back;
            if (!ok) flag(a.status, bad_any ? VELOX_STATUS_BAD_INDEX : VELOX_STATUS_NO_SPACE);
        }
    }
    for (int p = rank * PT + threadIdx.x; p < back; p += ctas * PT) {
        const int r = owner(pg, a.R, p);
        a.free_list[fc + p] = a.table[static_cast<long long>(r) * a.max_pages + p - pg[r]];
    }
}

int cluster_launch(void (*kern)(PlanArgs), const PlanArgs& a, int ctas, size_t smem,
                   cudaStream_t st) {
    if (cudaFuncSetAttribute(reinterpret_cast<const void*>(kern),
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem)) != cudaSuccess)
        return VELOX_ECUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(PT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ctas;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? VELOX_OK : VELOX_ECUDA;
}

}  // namespace

int paged_plan_launch(const PlanArgs& a, cudaStream_t st) {
    const int ctas = a.n_cap <= PT ? 1 : 8;
    return cluster_launch(paged_plan_kernel, a, ctas, sizeof(int) * 3 * (a.R + 1), st);
}

int paged_release_launch(const PlanArgs& a, cudaStream_t st) {
    const int ctas = static_cast<long long>(a.R) * a.max_pages <= PT ? 1 : 8;
    return cluster_launch(paged_release_kernel, a, ctas, sizeof(int) * (a.R + 1), st);
}

}  // namespace velox
