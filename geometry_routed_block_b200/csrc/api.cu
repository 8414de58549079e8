// C ABI of libvelox: argument validation, then kernel launches on the caller's
// stream. Nothing here allocates, frees or synchronises.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "velox_internal.cuh"

namespace {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }
inline bool tile_ok(int x) { return x == 64 || x == 128; }

}  // namespace

extern "C" {

int velox_version(void) { return 100; }

const char* velox_strerror(int code) {
    switch (code) {
        case VELOX_OK: return "ok";
        case VELOX_EINVAL: return "invalid argument";
        case VELOX_EUNSUPPORTED: return "unsupported configuration";
        case VELOX_ECUDA: return "CUDA error";
        case VELOX_ETIMEOUT: return "bounded wait expired";
        case VELOX_EBOUNDS: return "index out of range";
        default: return "unknown error";
    }
}

int velox_slices_build(const float* depth, const float* poses, const float* intr, int P, int Hp,
                       int Wp, velox_slice_t* slices, void* stream) {
    if (!depth || !poses || !intr || !slices || P < 1 || Hp < 1 || Wp < 1) return VELOX_EINVAL;
    return velox::slices_launch(depth, poses, intr, P, Hp * Wp, slices, as_stream(stream));
}

int velox_block_overlap(const float* cur_depth, const velox_slice_t* cur_cam,
                        const velox_slice_t* slices, int B, int P, int F, int Hp, int Wp, int T,
                        int32_t* counts, void* stream) {
    if (!cur_depth || !cur_cam || !slices || !counts) return VELOX_EINVAL;
    if (B < 1 || P < 1 || F < 1 || Hp < 1 || Wp < 1 || T < 32 || T > 1024 || (T % 32) != 0)
        return VELOX_EINVAL;
    const long long Nq = static_cast<long long>(F) * Hp * Wp;
    if (Nq % T != 0 || Nq > (1ll << 30)) return VELOX_EINVAL;
    const int m = static_cast<int>(Nq / T);
    return velox::overlap_launch(cur_depth, cur_cam, slices, B, P, Hp, Wp, T, m, counts,
                                 as_stream(stream));
}

size_t velox_route_topk_workspace_size(int B, int H, int Nq, int Nk, int d, int T) {
    if (B < 1 || H < 1 || T < 1 || Nq < T || Nq % T || Nk < Nq || Nk % Nq || d < 1) return 0;
    const int m = Nq / T;
    const int n_past = (Nk - Nq) / T;
    return velox::route_ws_bytes(B, H, m, n_past, d, T);
}

int velox_route_topk(const void* q, const void* k, int dtype, int B, int H, int Nq, int Nk, int d,
                     int T, const int32_t* counts, float alpha, int topk, int32_t* idx, void* ws,
                     size_t ws_bytes, void* counts_ready, void* stream) {
    if (!q || !k || !idx || !ws) return VELOX_EINVAL;
    if (dtype != VELOX_BF16 && dtype != VELOX_F32) return VELOX_EUNSUPPORTED;
    if (B < 1 || H < 1 || Nq < 1 || Nk < 1 || d < 1 || T < 1) return VELOX_EINVAL;
    if (!tile_ok(T) || !tile_ok(d)) return VELOX_EUNSUPPORTED;
    if (Nq % T || Nk % Nq) return VELOX_EINVAL;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(ws, 256) || !aligned(idx, 4))
        return VELOX_EINVAL;
    if (!std::isfinite(alpha)) return VELOX_EINVAL;
    const int m = Nq / T;
    const int n_kb = Nk / T;
    if (topk < m || topk > n_kb) return VELOX_EINVAL;
    const size_t need = velox_route_topk_workspace_size(B, H, Nq, Nk, d, T);
    if (need == 0 || ws_bytes < need) return VELOX_EINVAL;
    if (static_cast<long long>(B) * H * Nk * d >= (1ll << 40)) return VELOX_EINVAL;
    if (Nk / T > 8192) return VELOX_EINVAL;  // key-block index range of the selection

    velox::RouteArgs r{};
    r.B = B;
    r.H = H;
    r.Nq = Nq;
    r.Nk = Nk;
    r.d = d;
    r.T = T;
    r.m = m;
    r.P = Nk / Nq - 1;
    r.n_past = r.P * m;
    r.topk = topk;
    r.counts = r.P > 0 ? counts : nullptr;
    r.alpha = alpha;
    r.inv_sqrt_d = static_cast<float>(1.0 / std::sqrt(static_cast<double>(d)));
    r.idx = idx;
    const size_t rows = static_cast<size_t>(B) * H * m;
    const size_t qbar_bytes = (rows * d * sizeof(float) + 255) & ~static_cast<size_t>(255);
    r.qbar = static_cast<float*>(ws);
    r.scores = reinterpret_cast<float*>(static_cast<char*>(ws) + qbar_bytes);
    if (velox::route_split_scoring(T, d)) {
        const size_t scores_bytes =
            (rows * static_cast<size_t>(r.n_past) * sizeof(float) + 255) & ~static_cast<size_t>(255);
        r.kbar_ws = reinterpret_cast<float*>(static_cast<char*>(ws) + qbar_bytes + scores_bytes);
    }
    r.counts_ready = static_cast<cudaEvent_t>(counts_ready);
    return velox::route_launch(q, k, dtype, r, as_stream(stream));
}

}  // extern "C"

namespace {

int sparse_attn(const void* q, const void* k, const void* v, const int32_t* idx, int topk, int B,
                int H, int Nq, int Nk, int d, int T, float scale, void* o, float* lse,
                int32_t* status, unsigned long long wait_ns, int skip_mma, int force_pair,
                void* stream) {
    if (!q || !k || !v || !o) return VELOX_EINVAL;
    if (B < 1 || H < 1 || Nq < 1 || Nk < 1 || d < 1 || T < 1) return VELOX_EINVAL;
    if (!tile_ok(T) || !tile_ok(d)) return VELOX_EUNSUPPORTED;
    if (Nq % T || Nk % T) return VELOX_EINVAL;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16))
        return VELOX_EINVAL;
    if (!(scale > 0.0f) || !std::isfinite(scale)) return VELOX_EINVAL;
    const long long rows_k = static_cast<long long>(B) * H * Nk;
    if (rows_k >= (1ll << 31) || static_cast<long long>(B) * H * Nq >= (1ll << 31))
        return VELOX_EINVAL;
    const int n_kb = Nk / T;
    if (idx && (topk < 1 || topk > n_kb)) return VELOX_EINVAL;
    if (H > 65535 || B > 65535) return VELOX_EINVAL;

    velox::AttnArgs a{};
    a.idx = idx;
    a.n_sel = idx ? topk : n_kb;
    a.H = H;
    a.Nq = Nq;
    a.Nk = Nk;
    a.T = T;
    a.m = Nq / T;
    a.n_kb = n_kb;
    a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    a.o = static_cast<__nv_bfloat16*>(o);
    a.lse = lse;
    a.status = status;
    a.wait_ns = wait_ns;
    a.skip_mma = skip_mma;
    a.force_pair = force_pair;
    return velox::attn_fwd_launch(q, k, v, a, B, d, as_stream(stream));
}

}  // namespace

extern "C" {

int velox_sparse_attn_fwd(const void* q, const void* k, const void* v, const int32_t* idx,
                          int topk, int B, int H, int Nq, int Nk, int d, int T, float scale,
                          void* o, float* lse, int32_t* status, void* stream) {
    return sparse_attn(q, k, v, idx, topk, B, H, Nq, Nk, d, T, scale, o, lse, status,
                       velox::WAIT_LIMIT_NS, 0, 0, stream);
}

int velox_sparse_attn_fwd_test(const void* q, const void* k, const void* v, const int32_t* idx,
                               int topk, int B, int H, int Nq, int Nk, int d, int T, float scale,
                               void* o, float* lse, int32_t* status, double wait_limit_s,
                               int flags, void* stream) {
    if (!(wait_limit_s >= 1e-3 && wait_limit_s <= 10.0)) return VELOX_EINVAL;
    if (flags & ~(VELOX_TEST_SKIP_MMA | VELOX_TEST_FORCE_PAIR)) return VELOX_EINVAL;
    return sparse_attn(q, k, v, idx, topk, B, H, Nq, Nk, d, T, scale, o, lse, status,
                       static_cast<unsigned long long>(wait_limit_s * 1e9),
                       (flags & VELOX_TEST_SKIP_MMA) ? 1 : 0,
                       (flags & VELOX_TEST_FORCE_PAIR) ? 1 : 0, stream);
}

size_t velox_kbar_cache_bytes(int B, int H, int max_past_chunks, int Nq, int d, int T) {
    if (B < 1 || H < 1 || max_past_chunks < 1 || T < 1 || Nq < T || Nq % T || d < 1) return 0;
    return static_cast<size_t>(B) * H * max_past_chunks * (Nq / T) * d * sizeof(float);
}

int velox_kbar_append(const void* k, int dtype, int B, int H, int Nk, int Nq, int d, int T, int chunk,
                      float* kbar, int max_past_chunks, void* stream) {
    if (!k || !kbar) return VELOX_EINVAL;
    if (dtype != VELOX_BF16 && dtype != VELOX_F32) return VELOX_EUNSUPPORTED;
    if (B < 1 || H < 1 || Nq < 1 || Nk < 1 || d < 1 || T < 1 || max_past_chunks < 1)
        return VELOX_EINVAL;
    if (!tile_ok(T) || !tile_ok(d)) return VELOX_EUNSUPPORTED;
    if (Nq % T || Nk % T) return VELOX_EINVAL;
    if (chunk < 0 || chunk >= max_past_chunks || static_cast<long long>(chunk + 1) * Nq > Nk)
        return VELOX_EINVAL;
    if (!aligned(k, 16) || !aligned(kbar, 16)) return VELOX_EINVAL;
    if (static_cast<long long>(B) * H > 65535) return VELOX_EINVAL;
    return velox::kbar_append_launch(k, dtype, B * H, Nk, Nq, d, T, chunk, max_past_chunks * (Nq / T),
                                     kbar, as_stream(stream));
}

int velox_route_topk_cached(const void* q, int dtype, const float* kbar, int max_past_chunks, int B,
                            int H, int Nq, int P, int d, int T, const int32_t* counts, float alpha,
                            int topk, int32_t* idx, void* ws, size_t ws_bytes, void* counts_ready,
                            void* stream) {
    if (!q || !idx || !ws || (P > 0 && !kbar)) return VELOX_EINVAL;
    if (dtype != VELOX_BF16 && dtype != VELOX_F32) return VELOX_EUNSUPPORTED;
    if (B < 1 || H < 1 || Nq < 1 || d < 1 || T < 1 || P < 0 || P > max_past_chunks)
        return VELOX_EINVAL;
    if (!tile_ok(T) || !tile_ok(d)) return VELOX_EUNSUPPORTED;
    if (Nq % T) return VELOX_EINVAL;
    if (!aligned(q, 16) || !aligned(ws, 256) || !aligned(idx, 4) || (kbar && !aligned(kbar, 16)))
        return VELOX_EINVAL;
    if (!std::isfinite(alpha)) return VELOX_EINVAL;
    const long long Nk = static_cast<long long>(P + 1) * Nq;
    if (Nk >= (1ll << 31) || Nk / T > 8192) return VELOX_EINVAL;
    const int m = Nq / T;
    const int n_kb = static_cast<int>(Nk / T);
    if (topk < m || topk > n_kb) return VELOX_EINVAL;
    const size_t need = velox_route_topk_workspace_size(B, H, Nq, static_cast<int>(Nk), d, T);
    if (need == 0 || ws_bytes < need) return VELOX_EINVAL;

    velox::RouteArgs r{};
    r.B = B;
    r.H = H;
    r.Nq = Nq;
    r.Nk = static_cast<int>(Nk);
    r.d = d;
    r.T = T;
    r.m = m;
    r.P = P;
    r.n_past = P * m;
    r.topk = topk;
    r.counts = P > 0 ? counts : nullptr;
    r.alpha = alpha;
    r.inv_sqrt_d = static_cast<float>(1.0 / std::sqrt(static_cast<double>(d)));
    r.idx = idx;
    const size_t rows = static_cast<size_t>(B) * H * m;
    const size_t qbar_bytes = (rows * d * sizeof(float) + 255) & ~static_cast<size_t>(255);
    r.qbar = static_cast<float*>(ws);
    r.scores = reinterpret_cast<float*>(static_cast<char*>(ws) + qbar_bytes);
    r.counts_ready = static_cast<cudaEvent_t>(counts_ready);
    r.kbar = kbar;
    r.kbar_cap = max_past_chunks * m;
    return velox::route_launch(q, nullptr, dtype, r, as_stream(stream));
}

size_t velox_depth_multiwarp_workspace_size(int Hp, int Wp) {
    if (Hp < 1 || Wp < 1) return 0;
    return velox::multiwarp_ws_bytes(Hp * Wp);
}

int velox_depth_multiwarp(const float* past_depth, const velox_slice_t* past_cams,
                          const velox_slice_t* cur_cam, int P, int Hp, int Wp, float rel_tol,
                          float* cur_depth, void* ws, size_t ws_bytes, void* stream) {
    if (!past_depth || !past_cams || !cur_cam || !cur_depth || !ws) return VELOX_EINVAL;
    if (P < 1 || Hp < 1 || Wp < 1 || !(rel_tol >= 0.0f) || !std::isfinite(rel_tol))
        return VELOX_EINVAL;
    if (static_cast<long long>(P) * Hp * Wp >= (1ll << 31)) return VELOX_EINVAL;
    if (!aligned(ws, 8) || ws_bytes < velox_depth_multiwarp_workspace_size(Hp, Wp))
        return VELOX_EINVAL;
    return velox::multiwarp_launch(past_depth, past_cams, cur_cam, P, Hp, Wp, rel_tol, cur_depth,
                                   ws, as_stream(stream));
}

int velox_fp64_fma_bench(double* out, int blocks, int threads, int iters, void* stream) {
    if (!out || blocks < 1 || threads < 32 || threads > 1024 || (threads % 32) != 0 || iters < 1)
        return VELOX_EINVAL;
    return velox::fp64_fma_launch(out, blocks, threads, iters, as_stream(stream));
}

int velox_cast_bf16(const float* x, uint16_t* y, size_t n, void* stream) {
    if (!x || !y) return VELOX_EINVAL;
    if (n == 0) return VELOX_OK;
    return velox::cast_bf16_launch(x, y, n, as_stream(stream));
}

}  // extern "C"

namespace {

constexpr long long INT_LIMIT = 1ll << 31;
// heads of a rotary launch: the kernels count them in 32 bits, a part beyond the last
constexpr long long MAX_ROWS = 1ll << 30;

inline bool page_ok(int page) { return page == 16 || page == 32 || page == 64 || page == 128; }

inline int log2_page(int page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7; }

// Fills the rotation of a launch; `rope` may be NULL (nothing is rotated).
int set_rope(velox::RopeArgs& r, const velox_rope_t* rope, int d, const int32_t* pos) {
    if (!rope) {
        r.rot = 0;
        r.axes = 1;
        r.half_style = 1;
        return VELOX_OK;
    }
    if (rope->style != VELOX_ROPE_HALF && rope->style != VELOX_ROPE_INTERLEAVED)
        return VELOX_EUNSUPPORTED;
    if (rope->rot < 0 || rope->rot > d || rope->rot % 2 || rope->axes < 1 || rope->axes > 3)
        return VELOX_EINVAL;
    long long sum = 0;
    for (int i = 0; i < rope->axes; ++i) {
        if (rope->sections[i] < 0) return VELOX_EINVAL;
        sum += rope->sections[i];
    }
    if (sum != rope->rot / 2 || !std::isfinite(rope->mscale)) return VELOX_EINVAL;
    if (rope->rot > 0 && (!rope->freqs || !pos || !aligned(rope->freqs, 8) || !aligned(pos, 4)))
        return VELOX_EINVAL;
    r.rot = rope->rot;
    r.half_style = rope->style == VELOX_ROPE_HALF;
    r.axes = rope->axes;
    // first pair of axis 1 and of axis 2; an axis that is not there begins behind the last pair
    r.sec0 = rope->sections[0];
    r.sec01 = rope->axes > 1 ? rope->sections[0] + rope->sections[1] : rope->rot / 2;
    r.freqs = rope->freqs;
    r.pos = pos;
    r.mscale = rope->mscale;
    r.sign = rope->inverse ? -1.0f : 1.0f;
    return VELOX_OK;
}

// 16-byte accesses: every row starts on 16 bytes, and the rotated part and the rest are
// whole items of 8 elements
bool vec_rows(const void* p, int esize, int64_t s0, int64_t s1, int64_t s2) {
    const int64_t step = 16 / esize;
    return aligned(p, 16) && s0 % step == 0 && s1 % step == 0 && s2 % step == 0;
}
bool vec_rope(const velox::RopeArgs& r) {
    return r.d % 8 == 0 && r.rot % 8 == 0;
}

int paged_plan_check(const void* a, const void* b, const void* c, const void* d, const void* e,
                     const void* f, const void* g, int R, int max_pages, int page, int num_pages) {
    for (const void* p : {a, b, c, d, e, f, g})
        if (!p || !aligned(p, 4)) return VELOX_EINVAL;
    if (R < 1 || R > 8192 || page < 1 || max_pages < 1 || num_pages < 1) return VELOX_EINVAL;
    if (!page_ok(page)) return VELOX_EUNSUPPORTED;
    if (static_cast<long long>(max_pages) * page >= INT_LIMIT ||
        static_cast<long long>(num_pages) * page >= INT_LIMIT)
        return VELOX_EINVAL;
    return VELOX_OK;
}

// Checks and launch of the one-token attention. cu (may be null) and N: the rows of q.
int paged_attn_run(const void* q, const void* k_pages, const void* v_pages, const int32_t* table,
                   const int32_t* lens, const int32_t* cu, int R, int N, int H, int Hkv, int d,
                   int page, int num_pages, int max_pages, float scale, void* o, float* lse,
                   void* ws, size_t ws_bytes, int32_t* status, unsigned long long wait_ns,
                   int skip_warps, int most_cluster, void* stream) {
    if (!q || !k_pages || !v_pages || !table || !lens || !o) return VELOX_EINVAL;
    if (R < 1 || R > 65535 || N < 1 || Hkv < 1 || H < Hkv || H % Hkv || d < 1 || page < 1 ||
        num_pages < 1 || max_pages < 1)
        return VELOX_EINVAL;
    if (!tile_ok(d) || !page_ok(page)) return VELOX_EUNSUPPORTED;
    if (!aligned(q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(o, 16) ||
        !aligned(ws, 256) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(lse, 4) ||
        !aligned(cu, 4) || !aligned(status, 4))
        return VELOX_EINVAL;
    const float scale_log2 =
        static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    if (!(scale > 0.0f) || !std::isfinite(scale_log2)) return VELOX_EINVAL;
    // in this order no product leaves 63 bits
    if (static_cast<long long>(max_pages) * page >= INT_LIMIT ||
        static_cast<long long>(num_pages) * page >= INT_LIMIT ||
        static_cast<long long>(num_pages) * page * Hkv >= INT_LIMIT ||
        static_cast<long long>(R) * H >= INT_LIMIT || static_cast<long long>(N) * H >= INT_LIMIT)
        return VELOX_EINVAL;
    if (!velox::paged_attn_whole(R, H, Hkv, page, max_pages) &&
        (!ws || ws_bytes < velox::paged_attn_ws_bytes(R, H, Hkv, d)))
        return VELOX_EINVAL;

    velox::PagedAttnArgs a{};
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.table = table;
    a.lens = lens;
    a.cu = cu;
    a.N = N;
    a.R = R;
    a.H = H;
    a.Hkv = Hkv;
    a.page = page;
    a.page_shift = log2_page(page);
    a.num_pages = num_pages;
    a.max_pages = max_pages;
    a.scale_log2 = scale_log2;
    a.o = static_cast<__nv_bfloat16*>(o);
    a.lse = lse;
    a.part = static_cast<float*>(ws);
    a.status = status;
    a.wait_ns = wait_ns;
    a.skip_warps = skip_warps;
    a.most_cluster = most_cluster;
    return velox::paged_attn_launch(k_pages, v_pages, a, d, as_stream(stream));
}

}  // namespace

extern "C" {

int velox_rope_freqs(int rot, double base, int kind, double factor, int orig_len,
                     double beta_fast, double beta_slow, double* freqs, float* mscale) {
    if (!freqs || rot < 2 || rot % 2) return VELOX_EINVAL;
    if (kind < VELOX_ROPE_PLAIN || kind > VELOX_ROPE_BANDS) return VELOX_EUNSUPPORTED;
    if (!std::isfinite(base) || !(base > 1.0)) return VELOX_EINVAL;
    if (kind != VELOX_ROPE_PLAIN && (!std::isfinite(factor) || !(factor >= 1.0)))
        return VELOX_EINVAL;
    if (kind == VELOX_ROPE_BASE) {
        if (rot == 2) return VELOX_EINVAL;
        base *= std::pow(factor, static_cast<double>(rot) / (rot - 2));
        if (!std::isfinite(base)) return VELOX_EINVAL;
    }
    double low = 0.0, high = 1.0;
    if (kind == VELOX_ROPE_BANDS) {
        if (orig_len < 1 || !std::isfinite(beta_fast) || !(beta_slow > 0.0) ||
            !(beta_fast > beta_slow))
            return VELOX_EINVAL;
        // pair index that makes n turns over orig_len positions
        const auto index = [&](double n) {
            return rot * std::log(orig_len / (n * 6.283185307179586)) / (2.0 * std::log(base));
        };
        low = std::min(std::max(std::floor(index(beta_fast)), 0.0), rot - 1.0);
        high = std::min(std::max(std::ceil(index(beta_slow)), 0.0), rot - 1.0);
    }
    for (int i = 0; i < rot / 2; ++i) {
        const double f = std::pow(base, -2.0 * i / rot);
        double slow = 0.0;  // share of f / factor
        if (kind == VELOX_ROPE_LINEAR) slow = 1.0;
        if (kind == VELOX_ROPE_BANDS)
            slow = high > low ? std::min(std::max((i - low) / (high - low), 0.0), 1.0)
                              : (i > low ? 1.0 : 0.0);
        freqs[i] = slow == 0.0 ? f : f * (1.0 - slow) + f / factor * slow;
    }
    if (mscale)
        *mscale = kind == VELOX_ROPE_BANDS ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.0f;
    return VELOX_OK;
}

int velox_rope(const void* x, int dtype, int B, int H, int N, int d, const int64_t* xs,
               const int32_t* pos, int64_t pos_axis_stride, int64_t pos_batch_stride,
               const velox_rope_t* rope, void* y, const int64_t* ys, void* stream) {
    if (!x || !y || !rope || !xs || !ys) return VELOX_EINVAL;
    if (dtype != VELOX_BF16 && dtype != VELOX_F32) return VELOX_EUNSUPPORTED;
    if (B < 1 || H < 1 || H > MAX_ROWS || N < 1 || d < 1 || d > 4096) return VELOX_EINVAL;
    if (static_cast<long long>(B) * N >= INT_LIMIT) return VELOX_EINVAL;
    const int esize = dtype == VELOX_BF16 ? 2 : 4;
    if (!aligned(x, esize) || !aligned(y, esize)) return VELOX_EINVAL;
    const int dims[3] = {B, H, N};
    int64_t xd[3], yd[3];  // 0 along dimensions of size 1
    for (int i = 0; i < 3; ++i) {
        if (xs[i] < 0 || ys[i] < 0 || (ys[i] == 0 && dims[i] > 1)) return VELOX_EINVAL;
        xd[i] = dims[i] > 1 ? xs[i] : 0;
        yd[i] = dims[i] > 1 ? ys[i] : 0;
    }

    velox::RopeArgs r{};
    const int rc = set_rope(r, rope, d, pos);
    if (rc != VELOX_OK) return rc;
    r.groups = 1;
    r.rows = H;
    r.rotated_rows = r.rot > 0 ? H : 0;
    r.tokens = static_cast<long long>(B) * N;
    r.N = N;
    r.d = d;
    r.pos_axis = pos_axis_stride;
    r.pos_batch = pos_batch_stride;
    velox::RopeGroup& g = r.g[0];
    g.x = x;
    g.y = y;
    g.heads = H;
    g.rotate = 1;
    g.xb = xd[0], g.xh = xd[1], g.xn = xd[2];
    g.yb = yd[0], g.yh = yd[1], g.yn = yd[2];
    const bool vec = vec_rope(r) && vec_rows(x, esize, xd[0], xd[1], xd[2]) &&
                     vec_rows(y, esize, yd[0], yd[1], yd[2]);
    return velox::rope_launch(r, dtype, false, vec, as_stream(stream));
}

int velox_paged_append(const void* q, const void* k, const void* v, int dtype, int N, int H,
                       int Hkv, int d, const int64_t* qs, const int64_t* ks, const int64_t* vs,
                       const int32_t* slots, const int32_t* pos, int64_t pos_axis_stride,
                       const velox_rope_t* rope, void* q_out, void* k_pages, void* v_pages, int page,
                       int num_pages, int32_t* status, void* stream) {
    if (!k || !v || !ks || !vs || !slots || !k_pages || !v_pages) return VELOX_EINVAL;
    if ((q == nullptr) != (q_out == nullptr) || (q && !qs)) return VELOX_EINVAL;
    if (dtype != VELOX_BF16 && dtype != VELOX_F32) return VELOX_EUNSUPPORTED;
    if (N < 1 || Hkv < 1 || (q && H < 1) || d < 1 || page < 1 || num_pages < 1)
        return VELOX_EINVAL;
    if (!page_ok(page) || !tile_ok(d)) return VELOX_EUNSUPPORTED;
    const long long n_slots = static_cast<long long>(num_pages) * page;
    if (n_slots >= INT_LIMIT || static_cast<long long>(q ? H : 0) + 2ll * Hkv > MAX_ROWS)
        return VELOX_EINVAL;
    const int esize = dtype == VELOX_BF16 ? 2 : 4;
    if (!aligned(k, esize) || !aligned(v, esize) || (q && !aligned(q, esize))) return VELOX_EINVAL;
    if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || (q && !aligned(q_out, 16)) ||
        !aligned(slots, 4) || !aligned(status, 4))
        return VELOX_EINVAL;
    for (int i = 0; i < 2; ++i)
        if (ks[i] < 0 || vs[i] < 0 || (q && qs[i] < 0)) return VELOX_EINVAL;

    velox::RopeArgs r{};
    const int rc = set_rope(r, rope, d, pos);
    if (rc != VELOX_OK) return rc;
    r.tokens = N;
    r.N = N;
    r.d = d;
    r.pos_axis = pos_axis_stride;
    r.slots = slots;
    r.page = page;
    r.page_shift = log2_page(page);
    r.n_slots = n_slots;
    r.status = status;
    bool vec = vec_rope(r);
    const auto add = [&](const void* x, const int64_t* s, int heads, int rotate, void* y,
                         bool to_pages) {
        velox::RopeGroup& g = r.g[r.groups++];
        g.x = x;
        g.y = y;
        g.heads = heads;
        g.rotate = rotate;
        g.to_pages = to_pages;
        g.xn = N > 1 ? s[0] : 0, g.xh = heads > 1 ? s[1] : 0;
        g.yn = static_cast<long long>(heads) * d, g.yh = d;
        r.rows += heads;
        if (rotate) r.rotated_rows += heads;
        vec = vec && vec_rows(x, esize, g.xn, g.xh, 0);
    };
    const int rotate = r.rot > 0;
    if (q) add(q, qs, H, rotate, q_out, false);
    add(k, ks, Hkv, rotate, k_pages, true);
    add(v, vs, Hkv, 0, v_pages, true);
    return velox::rope_launch(r, dtype, true, vec, as_stream(stream));
}

int velox_paged_plan(const int32_t* add, const int32_t* lens, int32_t* table,
                     const int32_t* free_list, const int32_t* free_count, int R, int max_pages,
                     int page, int num_pages, int n_cap, int32_t* lens_out,
                     int32_t* free_count_out, int32_t* cu, int32_t* slots, int32_t* pos,
                     int32_t* req, int32_t* status, void* stream) {
    const int rc = paged_plan_check(add, lens, table, free_list, free_count, lens_out,
                                    free_count_out, R, max_pages, page, num_pages);
    if (rc != VELOX_OK) return rc;
    if (!cu || n_cap < 0 || (n_cap > 0 && !slots)) return VELOX_EINVAL;
    for (const void* p : {cu, slots, pos, req, status})
        if (!aligned(p, 4)) return VELOX_EINVAL;
    velox::PlanArgs a{};
    a.add = add;
    a.lens = lens;
    a.table = table;
    a.free_list = const_cast<int32_t*>(free_list);
    a.free_count = free_count;
    a.R = R;
    a.max_pages = max_pages;
    a.page_shift = log2_page(page);
    a.num_pages = num_pages;
    a.n_cap = n_cap;
    a.lens_out = lens_out;
    a.free_count_out = free_count_out;
    a.cu = cu;
    a.slots = slots;
    a.pos = pos;
    a.req = req;
    a.status = status;
    return velox::paged_plan_launch(a, as_stream(stream));
}

int velox_paged_release(const int32_t* done, const int32_t* lens, const int32_t* table,
                        int32_t* free_list, const int32_t* free_count, int R, int max_pages,
                        int page, int num_pages, int32_t* lens_out, int32_t* free_count_out,
                        int32_t* status, void* stream) {
    const int rc = paged_plan_check(done, lens, table, free_list, free_count, lens_out,
                                    free_count_out, R, max_pages, page, num_pages);
    if (rc != VELOX_OK) return rc;
    if (!aligned(status, 4)) return VELOX_EINVAL;
    velox::PlanArgs a{};
    a.add = done;
    a.lens = lens;
    a.table = const_cast<int32_t*>(table);
    a.free_list = free_list;
    a.free_count = free_count;
    a.R = R;
    a.max_pages = max_pages;
    a.page_shift = log2_page(page);
    a.num_pages = num_pages;
    a.lens_out = lens_out;
    a.free_count_out = free_count_out;
    a.status = status;
    return velox::paged_release_launch(a, as_stream(stream));
}

size_t velox_paged_attn_workspace_size(int R, int H, int Hkv, int d) {
    if (R < 1 || R > 65535 || Hkv < 1 || H < Hkv || H % Hkv || !tile_ok(d)) return 0;
    return velox::paged_attn_ws_bytes(R, H, Hkv, d);
}

int velox_paged_attn(const void* q, const void* k_pages, const void* v_pages, const int32_t* table,
                     const int32_t* lens, int R, int H, int Hkv, int d, int page, int num_pages,
                     int max_pages, float scale, void* o, float* lse, void* ws, size_t ws_bytes,
                     int32_t* status, void* stream) {
    return paged_attn_run(q, k_pages, v_pages, table, lens, nullptr, R, R, H, Hkv, d, page, num_pages,
                          max_pages, scale, o, lse, ws, ws_bytes, status, velox::WAIT_LIMIT_NS, 0,
                          velox::MAX_CLUSTER, stream);
}

int velox_paged_attn_step(const void* q, const void* k_pages, const void* v_pages,
                          const int32_t* table, const int32_t* lens, const int32_t* cu, int R, int N,
                          int H, int Hkv, int d, int page, int num_pages, int max_pages, float scale,
                          void* o, float* lse, void* ws, size_t ws_bytes, int32_t* status,
                          void* stream) {
    if (!cu) return VELOX_EINVAL;
    return paged_attn_run(q, k_pages, v_pages, table, lens, cu, R, N, H, Hkv, d, page, num_pages,
                          max_pages, scale, o, lse, ws, ws_bytes, status, velox::WAIT_LIMIT_NS, 0,
                          velox::MAX_CLUSTER, stream);
}

int velox_paged_attn_test(const void* q, const void* k_pages, const void* v_pages,
                          const int32_t* table, const int32_t* lens, int R, int H, int Hkv, int d,
                          int page, int num_pages, int max_pages, float scale, void* o, float* lse,
                          void* ws, size_t ws_bytes, int32_t* status, double wait_limit_s,
                          int skip_warps, int most_cluster, void* stream) {
    if (!(wait_limit_s >= 1e-3 && wait_limit_s <= 10.0)) return VELOX_EINVAL;
    if (skip_warps < 0 || skip_warps > 15 || most_cluster < 1 || most_cluster > velox::MAX_CLUSTER)
        return VELOX_EINVAL;
    return paged_attn_run(q, k_pages, v_pages, table, lens, nullptr, R, R, H, Hkv, d, page, num_pages,
                          max_pages, scale, o, lse, ws, ws_bytes, status,
                          static_cast<unsigned long long>(wait_limit_s * 1e9), skip_warps, most_cluster,
                          stream);
}

}  // extern "C"
