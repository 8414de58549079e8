// Internal declarations shared by the library's translation units.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/velox.h"

namespace velox {

// default limit of the attention kernels' bounded waits: 2 s, far above any
// legitimate wait
constexpr unsigned long long WAIT_LIMIT_NS = 2000000000ull;
constexpr int MAX_CLUSTER = 16;  // CTAs of a cluster

struct AttnArgs {
    const int32_t* idx;  // [B*H][m][n_sel] or nullptr (dense)
    int n_sel;           // key blocks per query block
    int H, Nq, Nk, T, m, n_kb;
    float scale_log2;    // softmax scale * log2(e)
    __nv_bfloat16* o;
    float* lse;
    int32_t* status;
    const __nv_bfloat16* q;  // set by the launcher
    long long q_rows;        // B * H * Nq
    unsigned long long wait_ns;  // limit of every bounded wait
    int skip_mma;                // test hook: the tensor-core issuer issues nothing
    int force_pair;              // test hook: d = T = 128 on the CTA-pair kernel
    int pair_tiles;              // set by the launcher: two 64-token blocks per 128-row tile
};

int attn_fwd_launch(const void* q, const void* k, const void* v, const AttnArgs& a, int B, int d,
                    cudaStream_t st);

int slices_launch(const float* depth, const float* poses, const float* intr, int P, int HW,
                  velox_slice_t* out, cudaStream_t st);
int overlap_launch(const float* depth, const velox_slice_t* cur, const velox_slice_t* slices, int B,
                   int P, int Hp, int Wp, int T, int m, int32_t* counts, cudaStream_t st);
size_t multiwarp_ws_bytes(int HW);
int multiwarp_launch(const float* past_depth, const velox_slice_t* past, const velox_slice_t* cur,
                     int P, int Hp, int Wp, float rel_tol, float* out, void* ws, cudaStream_t st);

struct RouteArgs {
    int B, H, Nq, Nk, d, T, m, P, n_past, topk;
    const int32_t* counts;
    float alpha, inv_sqrt_d;
    int32_t* idx;
    float* qbar;    // workspace [B*H*m][d]
    float* scores;  // workspace [B*H*m][n_past]
    cudaEvent_t counts_ready;  // selection waits for it when set
    const float* kbar;         // k-bar cache [B*H][kbar_cap][d], or nullptr: pool K here
    int kbar_cap;              // blocks per (b, h) in the cache
    float* kbar_ws;            // workspace [B*H][n_past][d] when the scoring is split, else nullptr
};
// Whether routing without a k-bar cache pools every past key block into the
// workspace first and scores from there (instead of scoring each block as it
// is pooled): for the block shapes whose scoring per byte of K would hold
// the stream back.
bool route_split_scoring(int T, int d);
size_t route_ws_bytes(int B, int H, int m, int n_past, int d, int T);
int route_launch(const void* q, const void* k, int dtype, const RouteArgs& r, cudaStream_t st);

int kbar_append_launch(const void* k, int dtype, int BH, int Nk, int Nq, int d, int T, int chunk,
                       int cap, float* kbar, cudaStream_t st);

// Rows of heads that a rotary launch handles: x is read, rotated (or only
// copied) and written to `y` (dense or strided) or, with `pages`, to the slots
// of a paged cache.
struct RopeGroup {
    const void* x;
    void* y;
    int heads;
    int rotate;
    int to_pages;
    long long xb, xh, xn;  // elements between batches, heads, tokens
    long long yb, yh, yn;  // the same of y (unused with to_pages)
};
struct RopeArgs {
    RopeGroup g[3];
    int groups;
    int rows;          // heads of all groups
    int rotated_rows;  // heads of the leading groups that are rotated
    long long tokens;
    int N;     // tokens per batch
    int d, rot, half_style, axes, sec0, sec01;
    const double* freqs;
    const int32_t* pos;
    long long pos_axis, pos_batch;
    float mscale, sign;
    const int32_t* slots;  // of the paged groups
    int page, page_shift;
    long long n_slots;
    int32_t* status;
};
// in_dtype / out_bf16 (else float32); vec: 16-byte accesses are possible throughout
int rope_launch(const RopeArgs& a, int in_dtype, bool out_bf16, bool vec, cudaStream_t st);

struct PlanArgs {
    const int32_t* add;   // plan: new tokens; release: requests that end
    const int32_t* lens;
    int32_t* table;
    int32_t* free_list;
    const int32_t* free_count;
    int R, max_pages, page_shift, num_pages, n_cap;
    int later;  // lengths and count are written by a kernel of their own
    int32_t* lens_out;
    int32_t* free_count_out;
    int32_t* cu;
    int32_t* slots;
    int32_t* pos;
    int32_t* req;
    int32_t* status;
};
int paged_plan_launch(const PlanArgs& a, cudaStream_t st);
int paged_release_launch(const PlanArgs& a, cudaStream_t st);

struct PagedAttnArgs {
    const __nv_bfloat16* q;
    const int32_t* table;
    const int32_t* lens;
    int R, H, Hkv, page, num_pages, max_pages;
    int group;       // query heads per key head
    int head_tiles;  // tiles of at most 16 query heads per key head
    int tile_heads;  // query heads per tile
    int grid;        // CTAs that share the work
    int page_shift;  // log2(page)
    int stages;      // units that a warp keeps in flight
    int whole_rows;  // CTAs per row where rows are not dealt out by length, else 0
    float scale_log2;
    __nv_bfloat16* o;
    float* lse;
    float* part;     // workspace: partial results
    int32_t* status;
    unsigned long long wait_ns;  // limit of every bounded wait
    int skip_warps;              // test hook: bit w: warp w of every CTA fetches nothing
    int most_cluster;            // CTAs of a cluster at most (test hook: fewer than the device's)
    int N;                       // rows of q and o
    const int32_t* cu;  // [R + 1]: first new token of each request; null: request r has row r
};
// CTAs per row where histories are so short that rows are not dealt out by length, and no
// workspace is needed; else 0
int paged_attn_whole(int R, int H, int Hkv, int page, int max_pages);
size_t paged_attn_ws_bytes(int R, int H, int Hkv, int d);
int paged_attn_launch(const void* k_pages, const void* v_pages, const PagedAttnArgs& a, int d,
                      cudaStream_t st);

int cast_bf16_launch(const float* x, uint16_t* y, size_t n, cudaStream_t st);
int fp64_fma_launch(double* out, int blocks, int threads, int iters, cudaStream_t st);

}  // namespace velox
