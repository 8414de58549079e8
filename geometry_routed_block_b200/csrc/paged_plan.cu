// Block tables and slot maps of a paged KV cache, built on the GPU from the
// requests' lengths, and pages given back.
//
// Per request r: need_r = ceil((lens+add)/page) - ceil(lens/page) pages. Their
// exclusive prefix sum P_r places them on the stack of free pages (request r's
// i-th new page is free_list[free_count - 1 - P_r - i]), that of `add` places
// its tokens. Integer work on a few kilobytes: what bounds it is latency, the
// launch and the chain lengths -> scan -> page ids -> slots. So every CTA scans all
// lengths by itself (8192 requests are 64 KB), keeps the prefix sums in shared
// memory and takes its part of the pages and of the tokens; a token's page comes from
// the free list where it is a new one, so that no CTA waits for another's table
// entries.
//
// The outputs may be the inputs (a captured step carries its state on), and then no
// CTA may write lengths before all have read them. One cluster of up to 8 CTAs does it
// with a cluster barrier in between; a larger grid leaves the state to a second, small
// kernel. In place, 64 requests: 8000 tokens 3.4 us in the cluster and 5.7 us with the second
// kernel, 16,000 tokens 4.7 and 5.9, 32,000 6.2 and 6.1, 64,000 9.3 and 6.3; 168,000
// tokens of 300 requests 5.5 us, in place 7.2.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "ptx.cuh"
#include "velox_internal.cuh"

namespace velox {

namespace {

constexpr int BIG = 1024, SMALL = 256;  // threads per CTA
constexpr int MAX_R = 8192;
constexpr int CLUSTER = 8;              // CTAs of a cluster

// as the rotary kernels: launches overlap, memory is touched in turn
__device__ __forceinline__ void take_turn() {
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// exclusive prefix over the CTA of two 64-bit values, and their totals; its barriers
// order what the threads wrote to shared memory before
template <int PT>
__device__ __forceinline__ void scan2(long long& a, long long& b, long long& ta, long long& tb,
                                      long long* sh) {
    constexpr int W = PT / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long x = a, y = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(~0u, x, o), v = __shfl_up_sync(~0u, y, o);
        if (lane >= o) x += u, y += v;
    }
    if (lane == 31) sh[warp] = x, sh[W + warp] = y;
    __syncthreads();
    if (warp == 0) {
        long long p = lane < W ? sh[lane] : 0, q = lane < W ? sh[W + lane] : 0;
#pragma unroll
        for (int o = 1; o < W; o <<= 1) {
            const long long u = __shfl_up_sync(~0u, p, o), v = __shfl_up_sync(~0u, q, o);
            if (lane >= o) p += u, q += v;
        }
        if (lane < W) sh[lane] = p, sh[W + lane] = q;
    }
    __syncthreads();
    ta = sh[W - 1], tb = sh[2 * W - 1];
    a = x - a + (warp ? sh[warp - 1] : 0);
    b = y - b + (warp ? sh[W + warp - 1] : 0);
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

// ceil(tokens / page); tokens below 2^31
__device__ __forceinline__ int pages_of(int tokens, int shift) {
    return static_cast<int>((static_cast<uint32_t>(tokens) + (1u << shift) - 1) >> shift);
}

__device__ __forceinline__ void flag(int32_t* status, int bit) {
    if (status) atomicOr(status, bit);
}

// shared memory: int tok[R + 1], pg[R + 1], old[R + 1]
template <int PT, bool ONE_CLUSTER>
__global__ void __launch_bounds__(PT) paged_plan_kernel(const __grid_constant__ PlanArgs a) {
    extern __shared__ int sm[];
    __shared__ long long sh[2 * PT / 32];
    __shared__ int bad_any;
    int* tok = sm;
    int* pg = tok + a.R + 1;
    int* old = pg + a.R + 1;
    const long long cap = static_cast<long long>(a.max_pages) << a.page_shift;
    const int per = (a.R + PT - 1) / PT;
    const int r0 = min(a.R, static_cast<int>(threadIdx.x) * per), r1 = min(a.R, r0 + per);

    take_turn();
    if (threadIdx.x == 0) bad_any = 0;
    const int fc = *a.free_count;
    // bit 0: a length that cannot be, bit 1: a request beyond its table row
    int bad = (fc < 0 || fc > a.num_pages) ? 1 : 0;
    long long nt = 0, np = 0;
    for (int r = r0; r < r1; ++r) {
        const int n = a.lens[r], m = a.add[r];
        old[r] = n, tok[r] = m;  // read once: what follows agrees with what was counted
        if (n < 0 || n > cap || m < 0) {
            bad |= 1;
            continue;
        }
        if (static_cast<long long>(n) + m > cap) {
            bad |= 2;
            continue;
        }
        nt += m;
        np += pages_of(n + m, a.page_shift) - pages_of(n, a.page_shift);
    }
    __syncthreads();
    if (bad) atomicOr(&bad_any, bad);
    long long t0 = nt, p0 = np, tt, tp;
    scan2<PT>(t0, p0, tt, tp, sh);
    const int worst = bad_any;
    const bool ok = worst == 0 && tp <= fc && tt <= a.n_cap;
    int tokens = 0, new_pages = 0;
    if (ok) {
        tokens = static_cast<int>(tt);
        new_pages = static_cast<int>(tp);
        int t = static_cast<int>(t0), p = static_cast<int>(p0);
        for (int r = r0; r < r1; ++r) {
            const int n = old[r], m = tok[r];
            tok[r] = t;
            pg[r] = p;
            t += m;
            p += pages_of(n + m, a.page_shift) - pages_of(n, a.page_shift);
        }
        if (threadIdx.x == 0) tok[a.R] = tokens, pg[a.R] = new_pages;
    }
    // every CTA has read the lengths and the count: they may be overwritten
    if (ONE_CLUSTER) cluster_sync();
    else __syncthreads();

    const int gtid = blockIdx.x * PT + threadIdx.x, all = gridDim.x * PT;
    if (blockIdx.x == 0) {
        for (int r = threadIdx.x; r < a.R; r += PT) {
            a.cu[r] = ok ? tok[r] : 0;
            if (!a.later) {
                if (ok) a.lens_out[r] = old[r] + tok[r + 1] - tok[r];
                else if (a.lens_out != a.lens) a.lens_out[r] = a.lens[r];
            }
        }
        if (threadIdx.x == 0) {
            a.cu[a.R] = tokens;
            if (!a.later) *a.free_count_out = fc - new_pages;
            if (!ok)
                flag(a.status, (worst & 1) ? VELOX_STATUS_BAD_INDEX : VELOX_STATUS_NO_SPACE);
        }
    }
    for (int p = gtid; p < new_pages; p += all) {
        const int r = owner(pg, a.R, p);
        const int col = pages_of(old[r], a.page_shift) + p - pg[r];
        a.table[static_cast<long long>(r) * a.max_pages + col] = a.free_list[fc - 1 - p];
    }
    bool stray = false;
    // unsigned: the step behind the last token may pass 2^31
    for (unsigned i = gtid; i < static_cast<unsigned>(a.n_cap); i += all) {
        const int t = static_cast<int>(i);
        int slot = -1, pos = -1, r = -1;
        if (t < tokens) {
            r = owner(tok, a.R, t);
            pos = old[r] + t - tok[r];
            const int col = pos >> a.page_shift, fresh = col - pages_of(old[r], a.page_shift);
            const int id = fresh < 0 ? a.table[static_cast<long long>(r) * a.max_pages + col]
                                     : a.free_list[fc - 1 - pg[r] - fresh];
            if (id >= 0 && id < a.num_pages)
                slot = (id << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
            else
                stray = true;
        }
        a.slots[t] = slot;
        if (a.pos) a.pos[t] = pos;
        if (a.req) a.req[t] = r;
    }
    if (stray) flag(a.status, VELOX_STATUS_BAD_INDEX);
}

// the new lengths and the new count of a plan whose grid could not write them: from cu,
// which is 0 throughout where the plan did not fit
__global__ void __launch_bounds__(BIG) paged_plan_commit_kernel(const __grid_constant__ PlanArgs a) {
    __shared__ long long sh[2 * BIG / 32];
    take_turn();
    const int fc = *a.free_count;
    int now[MAX_R / BIG];
    long long np = 0, none = 0, tp, tn;
#pragma unroll
    for (int i = 0; i < MAX_R / BIG; ++i) {
        const int r = threadIdx.x + i * BIG;
        if (r < a.R) {
            const int n = a.lens[r], m = a.cu[r + 1] - a.cu[r];
            now[i] = n + m;
            if (m > 0) np += pages_of(n + m, a.page_shift) - pages_of(n, a.page_shift);
        }
    }
    scan2<BIG>(np, none, tp, tn, sh);  // also: everything has been read
#pragma unroll
    for (int i = 0; i < MAX_R / BIG; ++i)
        if (threadIdx.x + i * BIG < a.R) a.lens_out[threadIdx.x + i * BIG] = now[i];
    if (threadIdx.x == 0) *a.free_count_out = fc - static_cast<int>(tp);
}

// Whether the pages of the requests that end (a.add != 0) can go back, how many they
// are (each request's own in count[], if given), and where this thread's requests (r0 ..
// r1 - 1) begin among them.
struct Back {
    int fc, pages, first;
    bool ok, bad;
};
template <int PT>
__device__ __forceinline__ Back count_back(const PlanArgs& a, int r0, int r1, long long* sh,
                                           int* bad_any, int* count) {
    const long long cap = static_cast<long long>(a.max_pages) << a.page_shift;
    if (threadIdx.x == 0) *bad_any = 0;
    Back k;
    k.fc = *a.free_count;
    int bad = (k.fc < 0 || k.fc > a.num_pages) ? 1 : 0;
    long long np = 0, none = 0, tp, tn;
    for (int r = r0; r < r1; ++r) {
        const int n = a.lens[r];
        const int c = n >= 0 && n <= cap && a.add[r] != 0 ? pages_of(n, a.page_shift) : 0;
        if (n < 0 || n > cap) bad = 1;
        if (count) count[r] = c;
        np += c;
    }
    __syncthreads();
    if (bad) *bad_any = 1;
    scan2<PT>(np, none, tp, tn, sh);
    k.bad = *bad_any != 0;
    k.ok = !k.bad && k.fc + tp <= a.num_pages;
    k.pages = k.ok ? static_cast<int>(tp) : 0;
    k.first = static_cast<int>(np);
    return k;
}

// shared memory: int pg[R + 1]
template <int PT, bool ONE_CLUSTER>
__global__ void __launch_bounds__(PT) paged_release_kernel(const __grid_constant__ PlanArgs a) {
    extern __shared__ int sm[];
    __shared__ long long sh[2 * PT / 32];
    __shared__ int bad_any;
    int* pg = sm;
    const int per = (a.R + PT - 1) / PT;
    const int r0 = min(a.R, static_cast<int>(threadIdx.x) * per), r1 = min(a.R, r0 + per);
    take_turn();
    const Back k = count_back<PT>(a, r0, r1, sh, &bad_any, pg);
    if (k.ok) {
        int p = k.first;
        for (int r = r0; r < r1; ++r) {
            const int c = pg[r];
            pg[r] = p;
            p += c;
        }
    }
    if (ONE_CLUSTER) cluster_sync();  // lengths and count read by every CTA
    else __syncthreads();

    if (blockIdx.x == 0) {
        if (!a.later)
            for (int r = threadIdx.x; r < a.R; r += PT)
                a.lens_out[r] = (k.ok && a.add[r] != 0) ? 0 : a.lens[r];
        if (threadIdx.x == 0) {
            if (!a.later) *a.free_count_out = k.fc + k.pages;
            if (!k.ok) flag(a.status, k.bad ? VELOX_STATUS_BAD_INDEX : VELOX_STATUS_NO_SPACE);
        }
    }
    for (int p = blockIdx.x * PT + threadIdx.x; p < k.pages; p += gridDim.x * PT) {
        const int r = owner(pg, a.R, p);
        a.free_list[k.fc + p] = a.table[static_cast<long long>(r) * a.max_pages + p - pg[r]];
    }
}

// the same for a release whose grid could not write lengths and count
__global__ void __launch_bounds__(BIG)
    paged_release_commit_kernel(const __grid_constant__ PlanArgs a) {
    __shared__ long long sh[2 * BIG / 32];
    __shared__ int bad_any;
    take_turn();
    const int per = (a.R + BIG - 1) / BIG;
    const int r0 = min(a.R, static_cast<int>(threadIdx.x) * per), r1 = min(a.R, r0 + per);
    const Back k = count_back<BIG>(a, r0, r1, sh, &bad_any, nullptr);
    for (int r = r0; r < r1; ++r) a.lens_out[r] = (k.ok && a.add[r] != 0) ? 0 : a.lens[r];
    if (threadIdx.x == 0) *a.free_count_out = k.fc + k.pages;
}

bool overlap(const int32_t* a, long long na, const int32_t* b, long long nb) {
    return a < b + nb && b < a + na;
}

int launch(void (*kern)(PlanArgs), const PlanArgs& a, int ctas, int threads, size_t smem,
           bool cluster, cudaStream_t st) {
    // static shared memory comes on top: raise the limit well before the default one
    if (smem > 40 * 1024 &&
        cudaFuncSetAttribute(reinterpret_cast<const void*>(kern),
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem)) != cudaSuccess)
        return VELOX_ECUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = ctas;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? VELOX_OK : VELOX_ECUDA;
}

// items: pages or tokens that the grid deals with, at most
int run(void (*small)(PlanArgs), void (*cluster)(PlanArgs), void (*big)(PlanArgs),
        void (*commit)(PlanArgs), PlanArgs a, long long items, size_t smem, cudaStream_t st) {
    const bool in_place = overlap(a.lens_out, a.R, a.lens, a.R) ||
                          overlap(a.lens_out, a.R, a.add, a.R) ||
                          overlap(a.free_count_out, 1, a.free_count, 1) ||
                          overlap(a.free_count_out, 1, a.lens, a.R) ||
                          overlap(a.lens_out, a.R, a.free_count, 1) ||
                          overlap(a.free_count_out, 1, a.add, a.R);
    a.later = 0;
    if (items <= BIG && a.R <= BIG) return launch(small, a, 1, SMALL, smem, false, st);
    const int ctas = static_cast<int>(std::min<long long>((items + BIG - 1) / BIG, 148));
    if (!in_place) return launch(big, a, ctas, BIG, smem, false, st);
    if (items <= 2 * CLUSTER * BIG)
        return launch(cluster, a, std::min(ctas, CLUSTER), BIG, smem, true, st);
    a.later = 1;
    const int rc = launch(big, a, ctas, BIG, smem, false, st);
    return rc != VELOX_OK ? rc : launch(commit, a, 1, BIG, 0, false, st);
}

}  // namespace

int paged_plan_launch(const PlanArgs& a, cudaStream_t st) {
    // every new page holds a new token
    return run(paged_plan_kernel<SMALL, false>, paged_plan_kernel<BIG, true>,
               paged_plan_kernel<BIG, false>, paged_plan_commit_kernel, a, std::max(a.n_cap, 1),
               sizeof(int) * 3 * (a.R + 1), st);
}

int paged_release_launch(const PlanArgs& a, cudaStream_t st) {
    const long long pages =
        std::min<long long>(a.num_pages, static_cast<long long>(a.R) * a.max_pages);
    return run(paged_release_kernel<SMALL, false>, paged_release_kernel<BIG, true>,
               paged_release_kernel<BIG, false>, paged_release_commit_kernel, a, pages,
               sizeof(int) * (a.R + 1), st);
}

}  // namespace velox
