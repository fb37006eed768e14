// evict_api.cu -- the extern "C" entry points for accumulated attention weight and
// eviction, of caches of key-value heads and of latent rows: argument checks on the host,
// and dispatch.
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "paged.h"

namespace kvd {
namespace {

kvd_status cuda_status(cudaError_t e) { return e == cudaSuccess ? KVD_OK : KVD_ERR_CUDA; }

// c is checked; max_heads: query heads a KV head.
kvd_status mass_call(const kvd_paged_cache &c, const kvd_heads *q, const float *lse,
                     int32_t n_tokens, const int32_t *starts, int32_t max_new, float softmax_scale,
                     int32_t window, const float *mass, int64_t mass_stride, float decay,
                     float *out, int64_t out_stride, int max_heads, void *stream) {
    if (n_tokens < 0 || max_new < 0 || window < 0) return KVD_ERR_INVALID;
    if (!std::isfinite(decay) || decay < 0.0f) return KVD_ERR_INVALID;
    if (!out || !aligned(out, 4) || out_stride < c.len || !aligned(mass, 4)) return KVD_ERR_INVALID;
    if (decay > 0.0f && (!mass || mass_stride < c.len)) return KVD_ERR_INVALID;
    if (mass == out && mass_stride != out_stride) return KVD_ERR_INVALID;
    MassArgs a = {};
    PagedAttnArgs &p = a.attn;
    p.c = c;
    if (n_tokens > 0 && max_new > 0) {
        const kvd_status s = check_rows(q, c.head_dim);
        if (s != KVD_OK) return s;
        if (q->n_heads % c.n_kv_heads != 0) return KVD_ERR_INVALID;
        if (q->dtype != KVD_X_F16 && q->dtype != KVD_X_BF16) return KVD_ERR_INVALID;
        if (c.dtype != KVD_INT8 && (c.dtype == KVD_BF16) != (q->dtype == KVD_X_BF16))
            return KVD_ERR_INVALID;
        if (!std::isfinite(softmax_scale) || !(softmax_scale > 0.0f)) return KVD_ERR_INVALID;
        if (q->n_heads / c.n_kv_heads > max_heads) return KVD_ERR_UNSUPPORTED;
        if (!starts || !aligned(starts, 4) || !lse || !aligned(lse, 16)) return KVD_ERR_INVALID;
        p.q = q->x;
        p.q_stride = q->stride;
        p.bf16 = q->dtype == KVD_X_BF16;
        p.G = q->n_heads / c.n_kv_heads;
        p.n_tokens = n_tokens;
        p.max_new = max_new;
        p.window = window < c.len ? window : 0;
        p.starts = starts;
        p.scale_log2 = softmax_scale * kLog2e;
        p.lse = const_cast<float *>(lse);
    }
    a.mass = decay > 0.0f ? mass : nullptr;
    a.out = out;
    a.mass_stride = mass_stride;
    a.out_stride = out_stride;
    a.decay = decay;
    return cuda_status(launch_mass(a, static_cast<cudaStream_t>(stream)));
}

kvd_status evict_call(const kvd_paged_cache &c, const float *mass, int64_t mass_stride,
                      int32_t keep, int32_t sink, int32_t recent, const int32_t *to,
                      int32_t to_cols, int32_t *kept, int32_t *lens_out, float *mass_out,
                      int64_t mass_out_stride, void *stream) {
    if (keep < 1 || sink < 0 || recent < 0 ||
        static_cast<int64_t>(sink) + recent > static_cast<int64_t>(keep))
        return KVD_ERR_INVALID;
    const int most = keep < c.len ? keep : c.len;
    if (!mass || !aligned(mass, 4) || mass_stride < c.len) return KVD_ERR_INVALID;
    if (!to || !aligned(to, 4) || to_cols < 1 ||
        static_cast<int64_t>(to_cols) * c.page_size < most)
        return KVD_ERR_INVALID;
    if (!kept || !aligned(kept, 4) || !lens_out || !aligned(lens_out, 4) || lens_out == c.seq_lens)
        return KVD_ERR_INVALID;
    if (!aligned(mass_out, 4) || (mass_out && (mass_out_stride < keep || mass_out == mass)))
        return KVD_ERR_INVALID;
    EvictArgs a = {};
    a.c = c;
    a.row_bytes = c.head_dim * (c.dtype == KVD_INT8 ? 1 : 2);
    if (c.dtype != KVD_INT8) a.c.k_scale = a.c.v_scale = nullptr;
    a.mass = mass;
    a.mass_stride = mass_stride;
    a.keep = keep;
    a.sink = sink;
    a.recent = recent;
    a.to = to;
    a.to_cols = to_cols;
    a.kept = kept;
    a.lens_out = lens_out;
    a.mass_out = mass_out;
    a.mass_out_stride = mass_out_stride;
    return cuda_status(launch_evict(a, static_cast<cudaStream_t>(stream)));
}

}  // namespace
}  // namespace kvd

using namespace kvd;

extern "C" {

kvd_status kvd_paged_mass(const kvd_paged_cache *cache, const kvd_heads *q, const float *lse,
                          int32_t n_tokens, const int32_t *starts, int32_t max_new,
                          float softmax_scale, int32_t window, const float *mass,
                          int64_t mass_stride, float decay, float *out, int64_t out_stride,
                          void *stream) {
    const kvd_status s = check_paged(cache);
    if (s != KVD_OK) return s;
    return mass_call(*cache, q, lse, n_tokens, starts, max_new, softmax_scale, window, mass,
                     mass_stride, decay, out, out_stride, 16, stream);
}

kvd_status kvd_latent_mass(const kvd_latent_cache *cache, const kvd_heads *q, const float *lse,
                           int32_t n_tokens, const int32_t *starts, int32_t max_new,
                           float softmax_scale, int32_t window, const float *mass,
                           int64_t mass_stride, float decay, float *out, int64_t out_stride,
                           void *stream) {
    const kvd_status s = check_latent(cache);
    if (s != KVD_OK) return s;
    return mass_call(latent_as_paged(*cache), q, lse, n_tokens, starts, max_new, softmax_scale,
                     window, mass, mass_stride, decay, out, out_stride, 1024, stream);
}

kvd_status kvd_paged_evict(const kvd_paged_cache *cache, const float *mass, int64_t mass_stride,
                           int32_t keep, int32_t sink, int32_t recent,
                           const int32_t *page_table_out, int32_t max_pages_out, int32_t *kept,
                           int32_t *seq_lens_out, float *mass_out, int64_t mass_out_stride,
                           void *stream) {
    const kvd_status s = check_paged(cache);
    if (s != KVD_OK) return s;
    return evict_call(*cache, mass, mass_stride, keep, sink, recent, page_table_out, max_pages_out,
                      kept, seq_lens_out, mass_out, mass_out_stride, stream);
}

kvd_status kvd_latent_evict(const kvd_latent_cache *cache, const float *mass, int64_t mass_stride,
                            int32_t keep, int32_t sink, int32_t recent,
                            const int32_t *page_table_out, int32_t max_pages_out, int32_t *kept,
                            int32_t *seq_lens_out, float *mass_out, int64_t mass_out_stride,
                            void *stream) {
    const kvd_status s = check_latent(cache);
    if (s != KVD_OK) return s;
    return evict_call(latent_as_paged(*cache), mass, mass_stride, keep, sink, recent,
                      page_table_out, max_pages_out, kept, seq_lens_out, mass_out,
                      mass_out_stride, stream);
}

}  // extern "C"
