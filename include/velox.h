/*
 * velox.h -- C ABI of libvelox, the B200 (sm_100a) implementation of the Velox
 * geometry-routed block-sparse attention path.
 *
 * The method (pages "Velox: Raumgedaechtnis beschleunigt Video-Weltmodelle",
 * section "Tiefenanalyse", and "Velox: 공간 메모리로 비디오 월드 모델 추론 가속",
 * sections "배경" and "심층 분석") routes each query token block of the current
 * chunk of a chunked video-diffusion world model to a subset of the key blocks
 * of the growing KV cache:
 *   1. every past chunk is a camera-frustum slice with a depth interval;
 *   2. the current chunk's depth comes from a recency-priority multiwarp of
 *      past depth into the current view;
 *   3. the overlap of a query block's 3D region with each past slice softly
 *      modulates the block importance the model computes itself; regions that
 *      no history covers get no geometric bias;
 *   4. routing happens at token-block granularity, the attention tile, so the
 *      kernel really skips the blocks it was not given.
 * The pages fix no formula; the readings implemented here are stated on each
 * entry point below.
 *
 * Conventions shared by every entry point
 *   - Every pointer argument is a DEVICE pointer owned by the caller unless
 *     stated otherwise. The library never allocates, frees or synchronises;
 *     scratch memory, where an operation needs it, is passed in by the caller
 *     (sizes from the matching *_workspace_size function). The one exception
 *     is velox_depth_multiwarp_noalloc, whose scratch is a fixed array owned
 *     by the library.
 *   - Tensors are dense, row-major, innermost dimension last. Q/K/V/O use the
 *     layout [B][H][N][d]. In the KV cache the past chunks come first (oldest
 *     first) and the current chunk occupies the last Nq keys.
 *   - Every call is asynchronous on `stream` (a cudaStream_t; NULL = legacy
 *     default stream): it validates its arguments, enqueues kernels and returns.
 *     A rejected call (VELOX_EINVAL / VELOX_EUNSUPPORTED) launches nothing.
 *   - Calls hold no global state and may run concurrently on distinct streams
 *     with distinct outputs and workspaces -- except velox_depth_multiwarp_noalloc:
 *     all its calls share the library's scratch array, so they must not
 *     overlap on the GPU (serialise them, e.g. on one stream).
 *   - `status` arguments (may be NULL) point to one device int32 that kernels
 *     OR VELOX_STATUS_* bits into when they detect a bad index, find no room or
 *     give up a bounded wait; the caller zeroes it and reads it back.
 */
#ifndef VELOX_H
#define VELOX_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define VELOX_API __attribute__((visibility("default")))
#else
#define VELOX_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* return codes */
#define VELOX_OK 0
#define VELOX_EINVAL (-1)       /* bad shape, null or misaligned pointer, topk out of range */
#define VELOX_EUNSUPPORTED (-2) /* valid request outside the compiled variants (T, d, dtype) */
#define VELOX_ECUDA (-3)        /* a CUDA runtime / driver call or kernel launch failed */
#define VELOX_ETIMEOUT (-4)     /* reported through the status word: a bounded wait expired */
#define VELOX_EBOUNDS (-5)      /* reported through the status word: an index was out of range */

/* status-word bits */
#define VELOX_STATUS_BAD_INDEX 1
#define VELOX_STATUS_TIMEOUT 2
#define VELOX_STATUS_NO_SPACE 4 /* velox_paged_plan / velox_paged_release: no room; nothing changed */

/* element types */
#define VELOX_BF16 0
#define VELOX_F32 1

/* A camera, and for a past chunk its frustum slice (72 bytes, float32).
 * R: world->camera rotation, row-major; x_c = R x_w + t. Camera axes follow
 * OpenCV (x right, y down, z forward); depth is z-depth (not ray length).
 * fx, fy, cx, cy: pinhole intrinsics in latent-grid pixel units; pixel (r, c)
 * has its centre at (c + 0.5, r + 0.5).
 * [znear, zfar]: closed depth interval of the slice; empty when znear > zfar
 * (the empty slice is [+inf, -inf]). Ignored where a call says so. */
typedef struct velox_slice_t {
    float R[9];
    float t[3];
    float fx, fy, cx, cy;
    float znear, zfar;
} velox_slice_t;

/* Library version (major*10000 + minor*100 + patch). */
VELOX_API int velox_version(void);

/* Human-readable text for a return code (static string, never NULL). */
VELOX_API const char* velox_strerror(int code);

/*
 * Frustum slices of past chunks (step 1 of "Tiefenanalyse": each past chunk is
 * a camera-frustum slice with a depth interval).
 *   depth  [P][Hp][Wp] float32  depth map of each past chunk (shared by its frames)
 *   poses  [P][12] float32      R (9, row-major) then t (3), world->camera
 *   intr   [P][4] float32       fx, fy, cx, cy
 *   slices [P] velox_slice_t    output
 * Reading: [znear, zfar] = [min, max] of the chunk's valid depth samples
 * (finite and > 0); a chunk with no valid sample gets the empty slice.
 * Errors: VELOX_EINVAL for P < 1, Hp < 1, Wp < 1 or a NULL pointer.
 */
VELOX_API int velox_slices_build(const float* depth, const float* poses, const float* intr, int P, int Hp,
                       int Wp, velox_slice_t* slices, void* stream);

/*
 * Query-block / past-slice overlap counts (steps 1 and 3 of "Tiefenanalyse";
 * region-level context choice of "배경").
 *   cur_depth [B][Hp][Wp] float32  current-chunk depth (NaN, inf or <= 0: no depth)
 *   cur_cam   [B] velox_slice_t    current camera (znear/zfar ignored)
 *   slices    [B][P] velox_slice_t past slices
 *   counts    [B][m][P] int32      output, m = F*Hp*Wp / T
 * Token tau of the current chunk (raster order frame, row, column) sits at the
 * centre of pixel (r, c) = ((tau mod Hp*Wp) / Wp, tau mod Wp) of the chunk's
 * depth map. It is back-projected with the current camera, moved into camera j
 * and counted for slice j when znear_j <= z <= zfar_j, z > 0 and its
 * projection lies in [0, Wp) x [0, Hp). Tokens without valid depth count as
 * outside. Geometry runs in float64 with a fixed operation order and no fused
 * multiply-add, so counts are exact and reproducible.
 * Errors: VELOX_EINVAL for non-positive sizes, F*Hp*Wp not a multiple of T,
 * or a NULL pointer.
 */
VELOX_API int velox_block_overlap(const float* cur_depth, const velox_slice_t* cur_cam,
                        const velox_slice_t* slices, int B, int P, int F, int Hp, int Wp, int T,
                        int32_t* counts, void* stream);

/* Bytes of scratch velox_route_topk needs for these sizes (0 on bad sizes):
 * q-bar (B*H*m*d floats) and the block scores (B*H*m*n_past floats); with
 * T = 64 also the pooled past keys (B*H*n_past*d floats), which that block
 * size scores from after pooling them all (see velox_route_topk). */
VELOX_API size_t velox_route_topk_workspace_size(int B, int H, int Nq, int Nk, int d, int T);

/*
 * Geometry-modulated block routing (step 3 of "Tiefenanalyse": the slice
 * overlap softly modulates the model's own block importance; step 4: regions
 * no history covers keep the model's own routing).
 *   q      [B][H][Nq][d], k [B][H][Nk][d]  dtype VELOX_BF16 or VELOX_F32
 *   counts [B][m][P] int32 from velox_block_overlap, or NULL (no geometry)
 *   idx    [B][H][m][topk] int32 output: selected key blocks, ascending
 *   ws     scratch of velox_route_topk_workspace_size bytes (256-B aligned)
 *   counts_ready  a cudaEvent_t or NULL. When set, only the final selection
 *          kernel waits for it (cudaStreamWaitEvent): pooling and scoring, which
 *          do not read the counts, run meanwhile -- so the geometry (slices,
 *          overlap) can be produced on another stream at the same time.
 * with m = Nq/T query blocks, P = Nk/Nq - 1 past chunks, n_past = P*m past key
 * blocks, and key block kb covering keys [kb*T, (kb+1)*T).
 * Readings implemented:
 *   s[qb][kb]  = mean_T(Q block qb) . mean_T(K block kb) / sqrt(d)   (fp32)
 *   s'[qb][kb] = s + alpha * counts[qb][kb / m] / T   if sum_j counts[qb][j] > 0
 *              = s                                    otherwise (no bias)
 *   per (b, h, qb): the m current-chunk blocks are always kept and the
 *   topk - m past blocks with the largest s' are added (equal s': the smaller
 *   kb first). topk counts the current blocks.
 * With T = 128 each key block is scored as it is pooled; with T = 64 (twice the
 * query blocks per byte of K) every past block is pooled into the workspace
 * first and scored from there. Both give bit-identical scores.
 * Errors: VELOX_EINVAL for sizes that are not multiples (Nq % T, Nk % Nq),
 * more than 8192 key blocks (Nk/T), topk < m or topk > Nk/T, ws_bytes too
 * small, NULL or misaligned (16 B) pointers; VELOX_EUNSUPPORTED for T not in
 * {64,128}, d not in {64,128}, or an unknown dtype.
 */
VELOX_API int velox_route_topk(const void* q, const void* k, int dtype, int B, int H, int Nq, int Nk, int d,
                     int T, const int32_t* counts, float alpha, int topk, int32_t* idx, void* ws,
                     size_t ws_bytes, void* counts_ready, void* stream);

/*
 * Block-sparse attention forward over the routed blocks (step 4 of
 * "Tiefenanalyse"; the kernel walks only the listed key blocks).
 *   q [B][H][Nq][d], k/v [B][H][Nk][d]  bf16
 *   idx  [B][H][m][topk] int32, or NULL for dense attention over all Nk/T blocks
 *   o    [B][H][Nq][d] bf16 output
 *   lse  [B][H][Nq] float32 output (natural log of the softmax denominator of
 *        the scaled scores), or NULL
 * For every query row i of block qb: O_i = sum_j softmax_j(scale * Q_i.K_j) V_j
 * over the keys j of the listed blocks (no mask inside blocks; a block listed
 * twice counts twice). Tensor cores (tcgen05, TMEM accumulators) compute
 * Q K^T and P V in bf16 with fp32 accumulation; the softmax runs online in fp32.
 * Out-of-range entries of idx are replaced by block 0 and flagged in *status
 * (VELOX_STATUS_BAD_INDEX); bounded internal waits flag VELOX_STATUS_TIMEOUT.
 * Errors: VELOX_EINVAL for Nq % T, Nk % T, topk outside [1, Nk/T] (when idx is
 * given), NULL or non-16-byte-aligned q/k/v/o; VELOX_EUNSUPPORTED for T or d
 * outside {64,128}; VELOX_ECUDA when a tensor map cannot be encoded or the
 * launch fails.
 */
VELOX_API int velox_sparse_attn_fwd(const void* q, const void* k, const void* v, const int32_t* idx,
                          int topk, int B, int H, int Nq, int Nk, int d, int T, float scale,
                          void* o, float* lse, int32_t* status, void* stream);

/* test-hook flags of velox_sparse_attn_fwd_test */
#define VELOX_TEST_SKIP_MMA 1
#define VELOX_TEST_FORCE_PAIR 2

/*
 * velox_sparse_attn_fwd with two test hooks for its failure path; not a step
 * of the method. Every wait inside the attention kernels is bounded: a wait
 * that runs out sets VELOX_STATUS_TIMEOUT in *status, the CTA's other waits
 * give up, copies already in flight are drained and the kernel returns, so
 * the device stays usable. This entry point lets a test reach that path
 * without a fault:
 *   wait_limit_s  limit of each bounded wait, in seconds, in [1e-3, 10]
 *                 (velox_sparse_attn_fwd uses 2 s);
 *   flags         VELOX_TEST_SKIP_MMA: the tensor-core issuer issues nothing,
 *                 so no MMA completion ever arrives and the waits on them run
 *                 out (no MMA is in flight when tensor memory is freed); the
 *                 output is left unwritten.
 *                 VELOX_TEST_FORCE_PAIR: for d = T = 128, run the CTA-pair
 *                 kernel (two SMs per MMA, the union of two blocks' lists
 *                 walked once) also for routed lists, which otherwise go to the
 *                 single-SM two-block kernel; lists of more than 2048 blocks
 *                 still go there. 0: a normal call.
 * Other arguments, results and errors are those of velox_sparse_attn_fwd;
 * VELOX_EINVAL also for a limit outside the range or an unknown flag.
 */
VELOX_API int velox_sparse_attn_fwd_test(const void* q, const void* k, const void* v,
                                         const int32_t* idx, int topk, int B, int H, int Nq,
                                         int Nk, int d, int T, float scale, void* o, float* lse,
                                         int32_t* status, double wait_limit_s, int flags,
                                         void* stream);

/*
 * Pooled-key cache (an incremental form of the routing's key pooling; the
 * block importance the model computes in each layer, "Tiefenanalyse" step 3,
 * only ever needs the mean of each past key block, and a past chunk's keys
 * never change once the chunk is done).
 * The cache holds, per (b, h), the mean of each T-token key block of up to
 * max_past_chunks chunks: kbar [B][H][max_past_chunks * m][d] float32, m = Nq/T.
 */
VELOX_API size_t velox_kbar_cache_bytes(int B, int H, int max_past_chunks, int Nq, int d, int T);

/*
 * Pools the m key blocks of chunk `chunk` (keys [chunk*Nq, (chunk+1)*Nq) of every
 * (b, h) of the KV cache k [B][H][Nk][d], dtype VELOX_BF16 or VELOX_F32) into
 * kbar[b][h][chunk*m + i][:]. Call it once per chunk, when the chunk is done.
 * The values are bit-identical to the pooling velox_route_topk does itself.
 * Errors: VELOX_EINVAL for sizes that are not multiples, chunk outside
 * [0, max_past_chunks), keys [chunk*Nq, (chunk+1)*Nq) beyond Nk, NULL or
 * misaligned (16 B) pointers; VELOX_EUNSUPPORTED as velox_route_topk.
 */
VELOX_API int velox_kbar_append(const void* k, int dtype, int B, int H, int Nk, int Nq, int d, int T,
                                int chunk, float* kbar, int max_past_chunks, void* stream);

/*
 * velox_route_topk with the past key blocks taken from the pooled-key cache
 * instead of K: P past chunks (P <= max_past_chunks, chunks 0..P-1 appended)
 * and the current chunk, Nk = (P + 1) * Nq. Same arguments, semantics,
 * workspace (velox_route_topk_workspace_size(B, H, Nq, (P+1)*Nq, d, T)) and
 * errors; the selected blocks equal velox_route_topk's on the same keys.
 */
VELOX_API int velox_route_topk_cached(const void* q, int dtype, const float* kbar,
                                      int max_past_chunks, int B, int H, int Nq, int P, int d, int T,
                                      const int32_t* counts, float alpha, int topk, int32_t* idx,
                                      void* ws, size_t ws_bytes, void* counts_ready, void* stream);

/* Bytes of scratch velox_depth_multiwarp needs (0 on bad sizes). */
VELOX_API size_t velox_depth_multiwarp_workspace_size(int Hp, int Wp);

/*
 * Recency-priority multiwarp (step 2 of "Tiefenanalyse": past depth is warped
 * into the current view and recent history takes precedence).
 *   past_depth [P][Hp][Wp] float32, past_cams [P] velox_slice_t (znear/zfar
 *   ignored), cur_cam [1] velox_slice_t, cur_depth [Hp][Wp] float32 output.
 * Every valid past pixel (finite, > 0) is back-projected with its own camera,
 * moved into the current camera and, when in front of it and on the grid,
 * splatted on the pixel that contains its projection (floor). Per target
 * pixel: z_min = nearest candidate depth; candidates with
 * z <= z_min * (1 + rel_tol) win; the most recent winning chunk (largest
 * index) gives its smallest depth, rounded to float32. No candidate: NaN.
 * Float64 geometry, fixed operation order, no fused multiply-add.
 * ws: scratch of velox_depth_multiwarp_workspace_size bytes (8-B aligned).
 * Errors: VELOX_EINVAL for non-positive sizes, rel_tol < 0, a small workspace
 * or NULL pointers.
 */
VELOX_API int velox_depth_multiwarp(const float* past_depth, const velox_slice_t* past_cams,
                          const velox_slice_t* cur_cam, int P, int Hp, int Wp, float rel_tol,
                          float* cur_depth, void* ws, size_t ws_bytes, void* stream);

/* Largest grid (Hp * Wp) velox_depth_multiwarp_noalloc accepts. */
#define VELOX_MULTIWARP_NOALLOC_MAX_PIXELS 65536

/*
 * velox_depth_multiwarp without a caller workspace. The pages have no
 * counterpart to this call; it exists for callers that cannot allocate device
 * memory -- e.g. a plugin whose host passes it only its input and output
 * buffers, or a latency-critical loop that must not call cudaMalloc, which can
 * synchronise the device. Arguments and results are those of
 * velox_depth_multiwarp, minus ws / ws_bytes. Nothing is allocated or freed:
 * the scratch (20 bytes per pixel) is a fixed array in the library's own
 * device memory, 1.25 MiB, held on every GPU that loads the library until the
 * process exits.
 *   - Hp * Wp above VELOX_MULTIWARP_NOALLOC_MAX_PIXELS returns VELOX_EINVAL and
 *     launches nothing.
 *   - The first call in a CUDA context (normally: the first call on a device,
 *     whose primary context the runtime uses) looks up the array's device
 *     address with that context current and caches it under the context's
 *     id; make that first call before any stream capture. A context created
 *     later for the same device (after cudaDeviceReset, say) gets its own
 *     lookup. A failed lookup returns VELOX_ECUDA.
 *   - Every call resets the scratch it uses before reading it, but all calls
 *     share one array: calls whose kernels overlap on the GPU (e.g. on two
 *     streams at once) race and give wrong depths. Serialise them.
 */
VELOX_API int velox_depth_multiwarp_noalloc(const float* past_depth,
                                            const velox_slice_t* past_cams,
                                            const velox_slice_t* cur_cam, int P, int Hp, int Wp,
                                            float rel_tol, float* cur_depth, void* stream);

/*
 * float32 -> bf16 (round to nearest even) for n elements; used where a
 * workload's Q/K/V arrive in float32 and the attention tiles take bf16.
 * Errors: VELOX_EINVAL for NULL pointers.
 */
VELOX_API int velox_cast_bf16(const float* x, uint16_t* y, size_t n, void* stream);

/*
 * ---- Tokens: rotary positions, and a paged cache read by one new token -----
 *
 * A chunked world model also handles single tokens (an action, a state, a
 * caption token per rollout) and several rollouts of different lengths at once.
 * These calls are the block-sparse path's counterpart for them: rotary positions
 * of Q and K, a KV cache in pages that many requests share, and the attention of
 * one new token per request over its own pages.
 *
 * The paged cache of one layer is k_pages / v_pages [num_pages][Hkv][page][d]
 * bf16 (a page holds the heads of `page` consecutive tokens of one request, head by
 * head, as the block-sparse path's cache holds a whole history). Request r's
 * token t lies in page table[r][t / page], row t % page; table is [R][max_pages]
 * int32, and entries behind a request's pages are neither read nor written. A token's
 * slot is page_id * page + row. Free pages are a stack: the first *free_count
 * entries of free_list [num_pages], taken from and returned to its end.
 */

/* pair layouts of velox_rope_t */
#define VELOX_ROPE_HALF 0        /* pair i = elements (i, i + rot/2) */
#define VELOX_ROPE_INTERLEAVED 1 /* pair i = elements (2i, 2i + 1) */

/* frequency scalings of velox_rope_freqs */
#define VELOX_ROPE_PLAIN 0  /* f_i = base^(-2i/rot) */
#define VELOX_ROPE_LINEAR 1 /* f_i / factor */
#define VELOX_ROPE_BASE 2   /* base * factor^(rot/(rot-2)) in place of base */
#define VELOX_ROPE_BANDS 3  /* by wavelength, see velox_rope_freqs */

/* A rotation, a HOST struct that the call reads before it returns.
 * Element pair i (of rot/2) of a token is turned by the angle
 * t = pos[axis(i)] * freqs[i]:  (a, b) -> mscale * (a cos t - b sin t, b cos t + a sin t),
 * or by -t when `inverse` is set (the rotation's transpose, so also its gradient).
 * The first sections[0] pairs take their position from axis 0, the next
 * sections[1] from axis 1, and so on: one axis for running text or action tokens,
 * frame, row and column for the tokens of a chunk. Elements from rot on pass
 * unchanged. Angles are formed in float64, whatever the position; the rotation
 * runs in float32 and is rounded once. */
typedef struct velox_rope_t {
    const double* freqs; /* DEVICE, [rot/2] radians per position */
    int rot;             /* rotated elements of a head: even, 0 <= rot <= d */
    int style;           /* VELOX_ROPE_HALF or VELOX_ROPE_INTERLEAVED */
    int axes;            /* 1 to 3 */
    int sections[3];     /* pairs of each axis, >= 0; the first `axes` sum to rot/2 */
    float mscale;
    int inverse;
} velox_rope_t;

/*
 * The frequencies of `rot` rotated elements (of one axis), for velox_rope_t.
 *   freqs  HOST, [rot/2] float64 output; mscale  HOST, 1 float output, or NULL
 * kind VELOX_ROPE_BANDS (contexts `factor` times the original one of orig_len
 * positions): a pair that turns at least beta_fast times over orig_len positions
 * keeps f_i, one that turns at most beta_slow times gets f_i / factor, and
 * in between the two are mixed linearly in the pair's index, from floor of the
 * (real) index with beta_fast turns to ceil of the one with beta_slow, both held
 * within [0, rot - 1]; *mscale = 0.1 ln(factor) + 1. Every other kind gives
 * *mscale = 1. orig_len and the betas are read for VELOX_ROPE_BANDS alone.
 * Runs on the host and launches nothing.
 * Errors: VELOX_EINVAL for odd or non-positive rot, base <= 1, factor < 1, NULL
 * freqs, VELOX_ROPE_BASE with rot = 2, for VELOX_ROPE_BANDS orig_len < 1 or
 * not beta_fast > beta_slow > 0, and for values that are not finite;
 * VELOX_EUNSUPPORTED for an unknown kind.
 */
VELOX_API int velox_rope_freqs(int rot, double base, int kind, double factor, int orig_len,
                               double beta_fast, double beta_slow, double* freqs, float* mscale);

/*
 * Rotary positions of a tensor.
 *   x, y  [B][H][N][d], dtype VELOX_BF16 or VELOX_F32; y may be x (with x's strides),
 *         and shares no element with it otherwise
 *   xs, ys  HOST, elements between batches, heads and tokens of x and y (the
 *         innermost dimension is dense); 0 is allowed in xs alone
 *   pos   int32; token n of batch b has position
 *         pos[a * pos_axis_stride + b * pos_batch_stride + n] on axis a
 * Any alignment is taken; rows whose pointers, strides, rot and d allow 16-byte
 * accesses are faster.
 * Errors: VELOX_EINVAL for non-positive sizes, B*N >= 2^31, H > 2^30, d > 4096,
 * negative strides (or 0 in ys along a dimension longer than 1), an inconsistent
 * velox_rope_t (NULL freqs with rot > 0, odd rot or rot > d, axes outside 1..3,
 * sections that do not sum to rot/2, mscale not finite), pointers not aligned to
 * their element, or NULL x, y, rope, xs, ys (or pos with rot > 0);
 * VELOX_EUNSUPPORTED for an unknown dtype or style.
 */
VELOX_API int velox_rope(const void* x, int dtype, int B, int H, int N, int d, const int64_t* xs,
                         const int32_t* pos, int64_t pos_axis_stride, int64_t pos_batch_stride,
                         const velox_rope_t* rope, void* y, const int64_t* ys, void* stream);

/*
 * Block tables and slot map of a step, from the requests' lengths.
 *   add   [R] int32     new tokens of each request (0: none)
 *   lens  [R] int32     tokens already cached
 *   table [R][max_pages] int32   the new pages are entered behind the old ones
 *   free_list [num_pages], free_count [1] int32   the free pages (a stack)
 *   lens_out [R], free_count_out [1] int32 outputs; may be lens (or add) and free_count.
 *         Apart from that the outputs (table and status among them) share nothing with other
 *         arguments
 *   cu    [R + 1] int32 output: request r's new tokens are cu[r] .. cu[r+1] - 1
 *   slots, pos, req [n_cap] int32 outputs: slot, position in its request and
 *         request of each new token, -1 from token cu[R] on; pos and req may be
 *         NULL, and slots where n_cap = 0
 * Request r gets ceil((lens+add)/page) - ceil(lens/page) pages, requests in
 * order, each from the end of the stack. free_list itself is not changed, so a step
 * whose outputs are not its inputs may be planned again. Nothing is read back:
 * the call can be captured and replayed.
 * A plan that does not fit (more pages than are free, more tokens than n_cap, a
 * request beyond max_pages pages) changes nothing: lens and free_count are
 * handed on, cu is 0, every slot, pos and req is -1, and VELOX_STATUS_NO_SPACE
 * is set. The same with VELOX_STATUS_BAD_INDEX for a negative add, lens outside
 * [0, max_pages * page] or free_count outside [0, num_pages]. A token whose
 * page id in table or free_list is outside [0, num_pages) gets slot -1 and sets
 * VELOX_STATUS_BAD_INDEX.
 * Errors: VELOX_EINVAL for R outside [1, 8192], n_cap < 0, page, max_pages or
 * num_pages < 1, max_pages * page or num_pages * page >= 2^31, or NULL or
 * misaligned (4 B) pointers; VELOX_EUNSUPPORTED for page not in {16, 32, 64, 128}.
 */
VELOX_API int velox_paged_plan(const int32_t* add, const int32_t* lens, int32_t* table,
                               const int32_t* free_list, const int32_t* free_count, int R,
                               int max_pages, int page, int num_pages, int n_cap,
                               int32_t* lens_out, int32_t* free_count_out, int32_t* cu,
                               int32_t* slots, int32_t* pos, int32_t* req, int32_t* status,
                               void* stream);

/*
 * Gives the pages of finished requests back.
 *   done [R] int32: non-zero where request r ends. Its pages are pushed on the
 *   stack (requests in order, pages in order) and its length becomes 0; the
 *   table keeps its entries, which nothing reads any more.
 * Other arguments as velox_paged_plan. When more than num_pages pages would be
 * free (a page given back twice) nothing changes and VELOX_STATUS_NO_SPACE is
 * set; lens outside [0, max_pages * page] or free_count outside [0, num_pages]:
 * nothing changes, VELOX_STATUS_BAD_INDEX. Errors as velox_paged_plan.
 */
VELOX_API int velox_paged_release(const int32_t* done, const int32_t* lens, const int32_t* table,
                                  int32_t* free_list, const int32_t* free_count, int R,
                                  int max_pages, int page, int num_pages, int32_t* lens_out,
                                  int32_t* free_count_out, int32_t* status, void* stream);

/*
 * Writes N new tokens into one layer's pages, rotated on the way.
 *   q [N][H][d] (or NULL), k, v [N][Hkv][d]  dtype VELOX_BF16 or VELOX_F32
 *   qs, ks, vs  HOST, elements between tokens and between heads (slices of a fused
 *         projection, or [H][N][d] tensors; the innermost dimension is dense)
 *   slots [N] int32     slot of each token; negative: the token is padding, its k
 *         and v are not written. No slot may be given twice
 *   pos   int32, axis a of token n at pos[a * pos_axis_stride + n]
 *   rope  rotation of q and k, or NULL (none: pos is not read)
 *   q_out [N][H][d] bf16 output (dense; NULL without q): every row is written. It may
 *         be q itself (dense bf16), and shares no element with q, k or v otherwise
 *   k_pages, v_pages [num_pages][Hkv][page][d] bf16; other rows stay as they are. They share
 *         nothing with each other or with the other arguments
 * Everything is rounded to bf16 once, after the rotation. A slot of
 * num_pages * page or more is skipped and sets VELOX_STATUS_BAD_INDEX.
 * Errors: VELOX_EINVAL for non-positive sizes, H + 2 Hkv > 2^30 (H counted with q),
 * num_pages * page >= 2^31, negative strides, an inconsistent rope (see
 * velox_rope), pages or q_out not 16-byte aligned, other arrays not aligned to their
 * element, NULL pointers, q without q_out or the reverse; VELOX_EUNSUPPORTED for
 * page not in {16, 32, 64, 128}, d not in {64, 128}, an unknown dtype or style.
 */
VELOX_API int velox_paged_append(const void* q, const void* k, const void* v, int dtype, int N,
                                 int H, int Hkv, int d, const int64_t* qs, const int64_t* ks,
                                 const int64_t* vs, const int32_t* slots, const int32_t* pos,
                                 int64_t pos_axis_stride, const velox_rope_t* rope, void* q_out,
                                 void* k_pages, void* v_pages, int page, int num_pages,
                                 int32_t* status, void* stream);

/* Bytes of scratch velox_paged_attn needs for these sizes (0 on bad sizes). */
VELOX_API size_t velox_paged_attn_workspace_size(int R, int H, int Hkv, int d);

/*
 * Attention of one new token per request over its pages.
 *   q [R][H][d] bf16 (the layout [B][H][1][d] of the block-sparse path);
 *   k_pages, v_pages [num_pages][Hkv][page][d] bf16, H a multiple of Hkv: query
 *   head h reads key head h / (H / Hkv)
 *   table [R][max_pages], lens [R] int32: request r attends to its first lens[r]
 *   tokens (its new token among them, once appended)
 *   o [R][H][d] bf16 output; lse [R][H] float32 output (natural log of the softmax
 *   denominator of the scaled scores) or NULL. They share nothing with the other arguments
 *   ws  scratch of velox_paged_attn_workspace_size bytes (256-B aligned); may be
 *       NULL (ws_bytes 0) for short histories of few rows: where for an n of 1, 2, 4 or
 *       8, max_pages * page <= 512 n and R * Hkv * ceil(H / Hkv / 16) * n <= 256
 * table and lens must not change during the call: results are then undefined (what is read
 * and written stays within the arguments).
 * A request of length 0 gets zeros, with lse = -inf; one whose scores are all -inf gets NaN, as
 * a softmax of them, also with lse = -inf. What lies in a page behind the
 * last token may be anything, NaN too. Scores and softmax statistics are
 * float32; probabilities enter the tensor-core product as the sum of two bf16.
 * The history of every (request, key head) is split evenly over the GPU and
 * joined in a fixed order: results do not change from call to call.
 * Page ids outside [0, num_pages) are replaced by page 0 and lens outside
 * [0, max_pages * page] by the nearer bound; both set VELOX_STATUS_BAD_INDEX.
 * An expired internal wait sets VELOX_STATUS_TIMEOUT (outputs then undefined; nothing else
 * is written).
 * Errors: VELOX_EINVAL for R < 1 or R > 65535, H < 1, H not a multiple of Hkv,
 * scale not positive or scale * log2(e) not finite in float32, max_pages or
 * num_pages < 1, max_pages * page or num_pages * Hkv * page >= 2^31, R * H >= 2^31,
 * ws_bytes too small, NULL or misaligned (16 B; ws 256 B; int32 and float arrays 4 B)
 * pointers; VELOX_EUNSUPPORTED for page not in {16, 32, 64, 128} or d not in {64, 128}.
 */
VELOX_API int velox_paged_attn(const void* q, const void* k_pages, const void* v_pages,
                               const int32_t* table, const int32_t* lens, int R, int H, int Hkv,
                               int d, int page, int num_pages, int max_pages, float scale,
                               void* o, float* lse, void* ws, size_t ws_bytes, int32_t* status,
                               void* stream);

/*
 * velox_paged_attn for the rows of a planned step, as velox_paged_append returns them.
 *   cu [R + 1] int32  velox_paged_plan's: request r's new tokens are rows cu[r] .. cu[r+1] - 1
 *   q, o [N][H][d] bf16, lse [N][H]
 * A request with new tokens attends with the last of them, row cu[r+1] - 1, to its first
 * lens[r] tokens. A request without any is idle: its length, table and pages are not looked
 * at. Rows of o and lse that no request attends with (padding, all but the last of several
 * new tokens) are left as they were. A request whose rows are not within [0, N), or end
 * before they begin, is left out and sets VELOX_STATUS_BAD_INDEX; where cu gives several
 * requests one row, what that row holds is undefined.
 * Other arguments, limits and errors as velox_paged_attn; VELOX_EINVAL also for NULL or
 * misaligned cu, N < 1 or N * H >= 2^31.
 */
VELOX_API int velox_paged_attn_step(const void* q, const void* k_pages, const void* v_pages,
                                    const int32_t* table, const int32_t* lens, const int32_t* cu,
                                    int R, int N, int H, int Hkv, int d, int page, int num_pages,
                                    int max_pages, float scale, void* o, float* lse, void* ws,
                                    size_t ws_bytes, int32_t* status, void* stream);

/*
 * Test entry point: velox_paged_attn with a chosen limit for its bounded waits (1e-3 to
 * 10 s; the copies in flight are waited for with the default limit) and, bit w of
 * skip_warps (0 to 15), without the loads of warp w of every CTA, whose wait then runs
 * out; most_cluster (1 to 16): as on a device that cannot place clusters of more CTAs for a
 * single request. Not for product use.
 */
VELOX_API int velox_paged_attn_test(const void* q, const void* k_pages, const void* v_pages,
                                    const int32_t* table, const int32_t* lens, int R, int H,
                                    int Hkv, int d, int page, int num_pages, int max_pages,
                                    float scale, void* o, float* lse, void* ws, size_t ws_bytes,
                                    int32_t* status, double wait_limit_s, int skip_warps,
                                    int most_cluster, void* stream);

/*
 * Measurement helper, not a step of the method: blocks x threads threads each
 * run `iters` rounds of 8 independent float64 fused multiply-adds (2 FLOP each:
 * blocks * threads * iters * 16 FLOP per call), the ceiling that the float64
 * geometry (velox_block_overlap) is compared with. `out` (one double, device)
 * is written only in a case that does not occur, so the work cannot be
 * optimised away. Errors: VELOX_EINVAL for NULL out, blocks < 1, threads not a
 * multiple of 32 in [32, 1024], iters < 1.
 */
VELOX_API int velox_fp64_fma_bench(double* out, int blocks, int threads, int iters, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* VELOX_H */
