// paged_api.cu -- the extern "C" entry points for positions and norms, the paged
// cache and attention over it: argument checks on the host, and dispatch.
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "paged.h"

namespace kvd {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

namespace {

size_t x_size(int dtype) { return dtype == KVD_X_F32 ? 4 : 2; }

// What every cache in pages has: the page table and the counts.
kvd_status check_pages(const kvd_paged_cache *c) {
    if (c->batch < 1 || c->n_kv_heads < 1 || c->n_pages < 1 || c->max_pages < 1)
        return KVD_ERR_INVALID;
    if (c->page_size < 1) return KVD_ERR_INVALID;
    if (c->page_size % 16 != 0) return KVD_ERR_UNSUPPORTED;
    if (c->len < 0 || c->len > static_cast<int64_t>(c->max_pages) * c->page_size)
        return KVD_ERR_INVALID;
    // tokens, key tiles and rows of the pool are counted in 31 bits
    if (c->len > (1 << 30) ||
        static_cast<__int128>(c->batch) * c->n_kv_heads * (c->len / 128 + 1) > 0x7fffffff)
        return KVD_ERR_UNSUPPORTED;
    if (static_cast<__int128>(c->n_pages) * c->n_kv_heads * c->page_size > 0x7fffffff)
        return KVD_ERR_UNSUPPORTED;
    if (!c->k || !aligned(c->k, 16)) return KVD_ERR_INVALID;
    if (!c->page_table || !aligned(c->page_table, 4) || !c->seq_lens || !aligned(c->seq_lens, 4))
        return KVD_ERR_INVALID;
    if (c->dev_status && !aligned(c->dev_status, 4)) return KVD_ERR_INVALID;
    return KVD_OK;
}

}  // namespace

kvd_status check_rows(const kvd_heads *h, int head_dim) {
    if (!h || !h->x || !aligned(h->x, 16)) return KVD_ERR_INVALID;
    if (h->dtype != KVD_X_F16 && h->dtype != KVD_X_BF16 && h->dtype != KVD_X_F32)
        return KVD_ERR_INVALID;
    if (h->n_heads < 1 || h->n_heads > 65535) return KVD_ERR_INVALID;
    if (h->stride < static_cast<int64_t>(h->n_heads) * head_dim) return KVD_ERR_INVALID;
    if (h->stride % static_cast<int64_t>(16 / x_size(h->dtype)) != 0) return KVD_ERR_INVALID;
    return KVD_OK;
}

// A rotation (NULL: none) and the norms' weights against a head dim.
kvd_status check_rope(const kvd_rope *r, int head_dim, const float *qw, const float *kw,
                      float eps) {
    if (r) {
        if (!r->freqs || !aligned(r->freqs, 8) || r->reserved != 0) return KVD_ERR_INVALID;
        if (r->interleaved != 0 && r->interleaved != 1) return KVD_ERR_INVALID;
        if (!std::isfinite(r->mscale)) return KVD_ERR_INVALID;
        if (r->rot_dim < 1 || r->rot_dim > head_dim) return KVD_ERR_INVALID;
        if (r->rot_dim % 16 != 0) return KVD_ERR_UNSUPPORTED;
    }
    if ((qw && !aligned(qw, 16)) || (kw && !aligned(kw, 16))) return KVD_ERR_INVALID;
    if ((qw || kw) && (!(eps >= 0.0f) || !std::isfinite(eps))) return KVD_ERR_INVALID;
    return KVD_OK;
}

kvd_status check_paged(const kvd_paged_cache *c) {
    if (!c) return KVD_ERR_INVALID;
    if (c->dtype == KVD_Q8_0 || c->dtype == KVD_Q4_0) return KVD_ERR_UNSUPPORTED;
    if (c->dtype != KVD_F16 && c->dtype != KVD_BF16 && c->dtype != KVD_INT8)
        return KVD_ERR_INVALID;
    if (c->batch < 1 || c->n_kv_heads < 1 || c->n_pages < 1 || c->max_pages < 1)
        return KVD_ERR_INVALID;
    if (c->head_dim != 64 && c->head_dim != 128) return KVD_ERR_UNSUPPORTED;
    const kvd_status s = check_pages(c);
    if (s != KVD_OK) return s;
    if (!c->v || !aligned(c->v, 16)) return KVD_ERR_INVALID;
    if (c->dtype == KVD_INT8 && (!c->k_scale || !c->v_scale || !aligned(c->k_scale, 16) ||
                                 !aligned(c->v_scale, 16)))
        return KVD_ERR_INVALID;
    return KVD_OK;
}

kvd_paged_cache latent_as_paged(const kvd_latent_cache &c) {
    kvd_paged_cache p = {};
    p.dtype = c.dtype;
    p.batch = c.batch;
    p.n_kv_heads = 1;
    p.head_dim = c.rank + c.rope_dim;
    p.n_pages = c.n_pages;
    p.page_size = c.page_size;
    p.max_pages = c.max_pages;
    p.len = c.len;
    p.k = c.rows;
    p.page_table = c.page_table;
    p.seq_lens = c.seq_lens;
    p.dev_status = c.dev_status;
    return p;
}

kvd_status check_latent(const kvd_latent_cache *c) {
    if (!c) return KVD_ERR_INVALID;
    if (c->dtype == KVD_INT8 || c->dtype == KVD_Q8_0 || c->dtype == KVD_Q4_0)
        return KVD_ERR_UNSUPPORTED;
    if (c->dtype != KVD_F16 && c->dtype != KVD_BF16) return KVD_ERR_INVALID;
    if (c->rank < 1 || c->rope_dim < 1) return KVD_ERR_INVALID;
    if (c->rank % 128 != 0 || c->rank > 512 || c->rope_dim % 16 != 0 || c->rope_dim > 64)
        return KVD_ERR_UNSUPPORTED;
    const kvd_paged_cache p = latent_as_paged(*c);
    return check_pages(&p);
}

namespace {

kvd_status cuda_status(cudaError_t e) { return e == cudaSuccess ? KVD_OK : KVD_ERR_CUDA; }

// Whether two row arrays are the same array, which may be worked on in place.
bool same_rows(const kvd_heads *a, const kvd_heads *b) {
    return a->x == b->x && a->stride == b->stride && a->dtype == b->dtype;
}

kvd_status check_pair(const kvd_heads *in, const kvd_heads *out, int head_dim) {
    kvd_status s = check_rows(in, head_dim);
    if (s != KVD_OK) return s;
    if ((s = check_rows(out, head_dim)) != KVD_OK) return s;
    if (in->n_heads != out->n_heads) return KVD_ERR_INVALID;
    if (in->x == out->x && !same_rows(in, out)) return KVD_ERR_INVALID;
    return KVD_OK;
}

bool few_rows(int G, int max_new) { return static_cast<int64_t>(G) * max_new <= kDecodeRows; }

size_t attn_ws(const kvd_paged_cache &c, int H, int max_new) {
    const int G = H / c.n_kv_heads;
    return few_rows(G, max_new) ? paged_decode_ws(G * max_new, c.head_dim)
                                : paged_attn_ws(c, H, max_new);
}

RowsIn rows_in(const kvd_heads *h) { return RowsIn{h->x, h->stride, h->n_heads}; }
RowsOut rows_out(const kvd_heads *h) { return RowsOut{h->x, h->stride, h->dtype}; }

kvd_status attn_call(const kvd_paged_cache *cache, const kvd_heads *q, int32_t n_tokens,
                     const int32_t *starts, int32_t max_new, float softmax_scale, int32_t window,
                     const kvd_heads *out, float *lse, void *workspace, size_t workspace_bytes,
                     void *stream) {
    kvd_status s = check_paged(cache);
    if (s != KVD_OK) return s;
    if (n_tokens < 0 || max_new < 0 || window < 0) return KVD_ERR_INVALID;
    if (n_tokens == 0 || max_new == 0) return KVD_OK;
    const int D = cache->head_dim;
    if ((s = check_pair(q, out, D)) != KVD_OK) return s;
    if (q->n_heads % cache->n_kv_heads != 0 || q->dtype != out->dtype || q->x == out->x)
        return KVD_ERR_INVALID;
    if (q->dtype != KVD_X_F16 && q->dtype != KVD_X_BF16) return KVD_ERR_INVALID;
    if (cache->dtype != KVD_INT8 && (cache->dtype == KVD_BF16) != (q->dtype == KVD_X_BF16))
        return KVD_ERR_INVALID;
    if (!std::isfinite(softmax_scale) || !(softmax_scale > 0.0f)) return KVD_ERR_INVALID;
    const int G = q->n_heads / cache->n_kv_heads;
    if (G > 16) return KVD_ERR_UNSUPPORTED;
    if (!starts || !aligned(starts, 4)) return KVD_ERR_INVALID;
    if (!workspace || !aligned(workspace, 256) ||
        workspace_bytes < attn_ws(*cache, q->n_heads, max_new))
        return KVD_ERR_WORKSPACE;
    PagedAttnArgs a = {};
    a.c = *cache;
    a.q = q->x;
    a.out = out->x;
    a.q_stride = q->stride;
    a.out_stride = out->stride;
    a.bf16 = q->dtype == KVD_X_BF16;
    a.G = G;
    a.n_tokens = n_tokens;
    a.max_new = max_new;
    a.window = window < cache->len ? window : 0;  // positions plus it stay in 31 bits
    a.starts = starts;
    a.scale_log2 = softmax_scale * kLog2e;
    a.lse = lse;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return cuda_status(few_rows(G, max_new) ? launch_paged_decode(a, workspace, st)
                                            : launch_paged_attn(a, workspace, st));
}

}  // namespace
}  // namespace kvd

using namespace kvd;

extern "C" {

kvd_status kvd_rope_freqs(int32_t rot_dim, double base, int32_t scaling, double factor,
                          double orig_len, double low, double high, uint64_t *freqs,
                          float *mscale) {
    if (!freqs || !mscale) return KVD_ERR_INVALID;
    if (rot_dim < 16 || rot_dim > 1024 || rot_dim % 16 != 0) return KVD_ERR_INVALID;
    if (!std::isfinite(base) || base <= 1.0) return KVD_ERR_INVALID;
    if (scaling < KVD_ROPE_NONE || scaling > KVD_ROPE_BANDS) return KVD_ERR_INVALID;
    const bool ends = scaling == KVD_ROPE_YARN || scaling == KVD_ROPE_BANDS;
    if (scaling == KVD_ROPE_NONE) factor = 1.0;
    if (!std::isfinite(factor) || factor < 1.0) return KVD_ERR_INVALID;
    if (ends) {
        if (low == 0.0 && high == 0.0) {
            low = 1.0;
            high = scaling == KVD_ROPE_YARN ? 32.0 : 4.0;
        }
        if (!std::isfinite(orig_len) || orig_len < 1.0) return KVD_ERR_INVALID;
        if (!(low >= 0.0) || !std::isfinite(high) || low >= high) return KVD_ERR_INVALID;
        if (scaling == KVD_ROPE_YARN && low == 0.0) return KVD_ERR_INVALID;  // its logarithm
    }
    constexpr double kTwoPi = 6.283185307179586476925;
    const double r = rot_dim;
    if (scaling == KVD_ROPE_NTK) base *= std::pow(factor, r / (r - 2.0));
    double lo = 0.0, hi = 0.0;
    if (scaling == KVD_ROPE_YARN) {
        // the channel that turns so many times in orig_len positions
        auto channel = [&](double turns) {
            return r * std::log(orig_len / (turns * kTwoPi)) / (2.0 * std::log(base));
        };
        lo = std::fmax(std::floor(channel(high)), 0.0);
        hi = std::fmin(std::ceil(channel(low)), r - 1.0);
    }
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / r);
        double keep = 1.0;
        if (scaling == KVD_ROPE_LINEAR) keep = 0.0;
        if (scaling == KVD_ROPE_YARN)
            keep = 1.0 - std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 0.001), 0.0), 1.0);
        if (scaling == KVD_ROPE_BANDS)
            keep = std::fmin(std::fmax((orig_len * f / kTwoPi - low) / (high - low), 0.0), 1.0);
        f = f * (keep + (1.0 - keep) / factor);
        freqs[i] = static_cast<uint64_t>(std::llround(f / kTwoPi * 0x1p64));  // f <= 1: below 2^62
    }
    *mscale = scaling == KVD_ROPE_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.0f;
    return KVD_OK;
}

kvd_status kvd_qk_norm_rope(const kvd_heads *q, const kvd_heads *q_out, const kvd_heads *k,
                            const kvd_heads *k_out, int32_t n_tokens, int32_t head_dim,
                            const int32_t *positions, const kvd_rope *rope,
                            const float *q_weight, const float *k_weight, float eps,
                            void *stream) {
    if (n_tokens < 0) return KVD_ERR_INVALID;
    if (head_dim < 16 || head_dim > 1024 || head_dim % 16 != 0) return KVD_ERR_UNSUPPORTED;
    if (n_tokens == 0) return KVD_OK;
    kvd_status s = check_pair(q, q_out, head_dim);
    if (s != KVD_OK) return s;
    if ((k == nullptr) != (k_out == nullptr)) return KVD_ERR_INVALID;
    if (k) {
        if ((s = check_pair(k, k_out, head_dim)) != KVD_OK) return s;
        if (k->dtype != q->dtype) return KVD_ERR_INVALID;
    }
    if ((s = check_rope(rope, head_dim, q_weight, k_weight, eps)) != KVD_OK) return s;
    if (rope && (!positions || !aligned(positions, 4))) return KVD_ERR_INVALID;
    RopeArgs a = {};
    a.q = rows_in(q);
    a.q_out = rows_out(q_out);
    if (k) {
        a.k = rows_in(k);
        a.k_out = rows_out(k_out);
    }
    a.q_weight = q_weight;
    a.k_weight = k ? k_weight : nullptr;
    a.eps = eps;
    a.head_dim = head_dim;
    a.inv_dim = 1.0f / static_cast<float>(head_dim);
    a.n_tokens = n_tokens;
    a.positions = positions;
    if (rope) a.rope = *rope;
    return cuda_status(launch_rope(a, q->dtype, static_cast<cudaStream_t>(stream)));
}

kvd_status kvd_paged_append(const kvd_paged_cache *cache, const kvd_heads *k, const kvd_heads *v,
                            int32_t n_tokens, const int32_t *starts, const kvd_rope *rope,
                            const float *k_weight, const kvd_heads *q, const kvd_heads *q_out,
                            const float *q_weight, float eps, void *stream) {
    kvd_status s = check_paged(cache);
    if (s != KVD_OK) return s;
    if (n_tokens < 0) return KVD_ERR_INVALID;
    if (n_tokens == 0) return KVD_OK;
    const int D = cache->head_dim;
    if ((s = check_rows(k, D)) != KVD_OK) return s;
    if ((s = check_rows(v, D)) != KVD_OK) return s;
    if (k->n_heads != cache->n_kv_heads || v->n_heads != cache->n_kv_heads ||
        k->dtype != v->dtype)
        return KVD_ERR_INVALID;
    if ((q == nullptr) != (q_out == nullptr)) return KVD_ERR_INVALID;
    if (q) {
        if ((s = check_pair(q, q_out, D)) != KVD_OK) return s;
        if (q->dtype != k->dtype) return KVD_ERR_INVALID;
    }
    if ((s = check_rope(rope, D, q_weight, k_weight, eps)) != KVD_OK) return s;
    if (!starts || !aligned(starts, 4)) return KVD_ERR_INVALID;
    RopeArgs a = {};
    a.k = rows_in(k);
    a.v = rows_in(v);
    if (q) {
        a.q = rows_in(q);
        a.q_out = rows_out(q_out);
    }
    a.q_weight = q ? q_weight : nullptr;
    a.k_weight = k_weight;
    a.eps = eps;
    a.head_dim = D;
    a.inv_dim = 1.0f / static_cast<float>(D);
    a.n_tokens = n_tokens;
    if (rope) a.rope = *rope;
    a.starts = starts;
    a.cache = *cache;
    return cuda_status(launch_rope(a, k->dtype, static_cast<cudaStream_t>(stream)));
}

size_t kvd_paged_workspace_bytes(const kvd_paged_cache *cache, int32_t n_heads, int32_t n_tokens,
                                 int32_t max_new) {
    if (check_paged(cache) != KVD_OK || n_tokens < 1 || max_new < 1) return 0;
    if (n_heads < 1 || n_heads % cache->n_kv_heads != 0 || n_heads / cache->n_kv_heads > 16)
        return 0;
    return attn_ws(*cache, n_heads, max_new);
}

kvd_status kvd_paged_attn(const kvd_paged_cache *cache, const kvd_heads *q, int32_t n_tokens,
                          const int32_t *starts, int32_t max_new, float softmax_scale,
                          int32_t window, const kvd_heads *out, void *workspace,
                          size_t workspace_bytes, void *stream) {
    return attn_call(cache, q, n_tokens, starts, max_new, softmax_scale, window, out, nullptr,
                     workspace, workspace_bytes, stream);
}

kvd_status kvd_paged_attn_lse(const kvd_paged_cache *cache, const kvd_heads *q, int32_t n_tokens,
                              const int32_t *starts, int32_t max_new, float softmax_scale,
                              int32_t window, const kvd_heads *out, float *lse, void *workspace,
                              size_t workspace_bytes, void *stream) {
    // (without rows the call is a no-op, and an empty lse may be NULL)
    if (n_tokens != 0 && max_new != 0 && (!lse || !aligned(lse, 16))) return KVD_ERR_INVALID;
    return attn_call(cache, q, n_tokens, starts, max_new, softmax_scale, window, out, lse,
                     workspace, workspace_bytes, stream);
}

}  // extern "C"
