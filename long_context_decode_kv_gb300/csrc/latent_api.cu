// latent_api.cu -- the extern "C" entry points for the cache of latent rows: argument
// checks on the host, and dispatch.
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "paged.h"

namespace kvd {
namespace {

kvd_status cuda_status(cudaError_t e) { return e == cudaSuccess ? KVD_OK : KVD_ERR_CUDA; }

constexpr int kMaxHeads = 1024;

kvd_status check_parts(const kvd_head_parts *h, int channels) {
    if (!h || !h->x || !aligned(h->x, 16)) return KVD_ERR_INVALID;
    if (h->dtype != KVD_X_F16 && h->dtype != KVD_X_BF16 && h->dtype != KVD_X_F32)
        return KVD_ERR_INVALID;
    const int64_t unit = h->dtype == KVD_X_F32 ? 4 : 8;  // elements of 16 bytes
    if (h->n_heads < 1 || h->n_heads > 65535) return KVD_ERR_INVALID;
    if (h->head_stride < channels || h->head_stride > (1ll << 40) || h->head_stride % unit != 0 ||
        h->stride % unit != 0)
        return KVD_ERR_INVALID;
    if (h->stride < (h->n_heads - 1) * h->head_stride + channels) return KVD_ERR_INVALID;
    return KVD_OK;
}

}  // namespace
}  // namespace kvd

using namespace kvd;

extern "C" {

kvd_status kvd_latent_append(const kvd_latent_cache *cache, const kvd_heads *c,
                             const kvd_heads *k_pe, int32_t n_tokens, const int32_t *starts,
                             const kvd_rope *rope, const float *c_weight, const kvd_head_parts *q,
                             const kvd_head_parts *q_out, float eps, void *stream) {
    kvd_status s = check_latent(cache);
    if (s != KVD_OK) return s;
    if (n_tokens < 0) return KVD_ERR_INVALID;
    if (n_tokens == 0) return KVD_OK;
    if ((s = check_rows(c, cache->rank)) != KVD_OK) return s;
    if ((s = check_rows(k_pe, cache->rope_dim)) != KVD_OK) return s;
    if (c->n_heads != 1 || k_pe->n_heads != 1 || c->dtype != k_pe->dtype) return KVD_ERR_INVALID;
    if ((q == nullptr) != (q_out == nullptr)) return KVD_ERR_INVALID;
    if (q) {
        if ((s = check_parts(q, cache->rope_dim)) != KVD_OK) return s;
        if ((s = check_parts(q_out, cache->rope_dim)) != KVD_OK) return s;
        if (q->n_heads != q_out->n_heads || q->dtype != c->dtype) return KVD_ERR_INVALID;
        if (q->x == q_out->x && (q->stride != q_out->stride || q->head_stride != q_out->head_stride ||
                                 q->dtype != q_out->dtype))
            return KVD_ERR_INVALID;
    }
    if ((s = check_rope(rope, cache->rope_dim, c_weight, nullptr, eps)) != KVD_OK) return s;
    if (!starts || !aligned(starts, 4)) return KVD_ERR_INVALID;
    LatentAppendArgs a = {};
    a.c = RowsIn{c->x, c->stride, 1};
    a.k_pe = RowsIn{k_pe->x, k_pe->stride, 1};
    if (q) {
        a.q = RowsIn{q->x, q->stride, q->n_heads};
        a.q_head = q->head_stride;
        a.q_out = RowsOut{q_out->x, q_out->stride, q_out->dtype};
        a.q_out_head = q_out->head_stride;
    }
    a.c_weight = c_weight;
    a.eps = eps;
    a.inv_rank = 1.0f / static_cast<float>(cache->rank);
    a.rank = cache->rank;
    a.rope_dim = cache->rope_dim;
    a.n_tokens = n_tokens;
    if (rope) a.rope = *rope;
    a.starts = starts;
    a.cache = latent_as_paged(*cache);
    return cuda_status(launch_latent_append(a, c->dtype, static_cast<cudaStream_t>(stream)));
}

size_t kvd_latent_workspace_bytes(const kvd_latent_cache *cache, int32_t n_heads,
                                  int32_t n_tokens, int32_t max_new) {
    if (check_latent(cache) != KVD_OK || n_tokens < 1 || max_new < 1) return 0;
    if (n_heads < 1 || n_heads > kMaxHeads) return 0;
    return latent_attn_ws(n_heads, cache->rank, max_new);
}

kvd_status kvd_latent_attn(const kvd_latent_cache *cache, const kvd_heads *q, int32_t n_tokens,
                           const int32_t *starts, int32_t max_new, float softmax_scale,
                           int32_t window, const kvd_heads *out, float *lse, void *workspace,
                           size_t workspace_bytes, void *stream) {
    kvd_status s = check_latent(cache);
    if (s != KVD_OK) return s;
    if (n_tokens < 0 || max_new < 0 || window < 0) return KVD_ERR_INVALID;
    if (n_tokens == 0 || max_new == 0) return KVD_OK;
    if ((s = check_rows(q, cache->rank + cache->rope_dim)) != KVD_OK) return s;
    if ((s = check_rows(out, cache->rank)) != KVD_OK) return s;
    if (q->n_heads != out->n_heads || q->dtype != out->dtype || q->x == out->x)
        return KVD_ERR_INVALID;
    if (q->dtype != (cache->dtype == KVD_BF16 ? KVD_X_BF16 : KVD_X_F16)) return KVD_ERR_INVALID;
    if (q->n_heads > kMaxHeads) return KVD_ERR_UNSUPPORTED;
    if (!std::isfinite(softmax_scale) || !(softmax_scale > 0.0f)) return KVD_ERR_INVALID;
    if (!starts || !aligned(starts, 4) || (lse && !aligned(lse, 16))) return KVD_ERR_INVALID;
    if (!workspace || !aligned(workspace, 256) ||
        workspace_bytes < latent_attn_ws(q->n_heads, cache->rank, max_new))
        return KVD_ERR_WORKSPACE;
    PagedAttnArgs a = {};
    a.c = latent_as_paged(*cache);
    a.q = q->x;
    a.out = out->x;
    a.q_stride = q->stride;
    a.out_stride = out->stride;
    a.bf16 = q->dtype == KVD_X_BF16;
    a.G = q->n_heads;
    a.n_tokens = n_tokens;
    a.max_new = max_new;
    a.window = window < cache->len ? window : 0;  // positions plus it stay in 31 bits
    a.starts = starts;
    a.scale_log2 = softmax_scale * kLog2e;
    a.lse = lse;
    return cuda_status(
        launch_latent_attn(a, cache->rank, workspace, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
