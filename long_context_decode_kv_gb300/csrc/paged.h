// paged.h -- launchers of the kernels around a cache in pages for their C-ABI front ends:
// norm/rotation, append and attention (rope.cu, paged_attn.cu, paged_decode.cu, for
// paged_api.cu), latent rows (latent.cu, latent_attn.cu, for latent_api.cu), accumulated
// weights and eviction (mass.cu, evict.cu, for evict_api.cu).
// Arguments are already validated by the caller.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kvdecode.h"

namespace kvd {

// One launch of the norm/rotation kernel.  Heads of a token are numbered
// q, then k, then v; an absent part has zero heads.
struct RowsIn {
    const void *x;
    int64_t stride;
    int n_heads;
};
struct RowsOut {
    void *x;
    int64_t stride;
    int dtype;  // kvd_x_dtype
};
struct RopeArgs {
    RowsIn q, k, v;
    RowsOut q_out, k_out;  // k_out: unused with a cache
    const float *q_weight, *k_weight;
    float eps, inv_dim;  // inv_dim: 1 / head_dim
    int head_dim, n_tokens;
    const int32_t *positions;  // without a cache
    kvd_rope rope;             // rot_dim 0: no rotation
    const int32_t *starts;     // with a cache
    kvd_paged_cache cache;     // page_table NULL: no cache
};

cudaError_t launch_rope(const RopeArgs &a, int x_dtype, cudaStream_t st);

// One attention call.
struct PagedAttnArgs {
    kvd_paged_cache c;
    const void *q;
    void *out;
    int64_t q_stride, out_stride;
    bool bf16;  // q and out: bf16, else f16
    int G, n_tokens, max_new, window;
    const int32_t *starts;
    float scale_log2;  // softmax_scale * log2(e)
    float *lse;        // [n_tokens][heads] or NULL
};

// The workspace begins with paged_counter_bytes() of counters, zero between calls,
// which launch_paged_decode uses and launch_paged_attn leaves alone.
size_t paged_counter_bytes();
cudaError_t launch_paged_attn(const PagedAttnArgs &a, void *ws, cudaStream_t st);
size_t paged_attn_ws(const kvd_paged_cache &c, int H, int max_new);
// At most kDecodeRows rows (new tokens times query heads of a KV head) a sequence.
// Against the kernel for row tiles: one token over 512 f16 tokens 8.2 us and 17.9, 32
// rows over 8 int8 sequences of 131,072 605 us and 776.  The limit is not the best for
// f16: 32 rows over 8 sequences take 654 us and 617, 16 rows over one sequence of 32,764
// 56 and 40, and 32 over 32,768 85 and 41.
constexpr int kDecodeRows = 32;
cudaError_t launch_paged_decode(const PagedAttnArgs &a, void *ws, cudaStream_t st);
size_t paged_decode_ws(int rows, int D);

// Latent rows.  The cache is a kvd_paged_cache with one KV head of rank + rope_dim
// channels, its rows in k, and no v.
struct LatentAppendArgs {
    RowsIn c, k_pe, q;  // q: zero heads where there are none
    int64_t q_head;     // elements from one head of q to the next
    RowsOut q_out;
    int64_t q_out_head;
    const float *c_weight;
    float eps, inv_rank;
    int rank, rope_dim, n_tokens;
    kvd_rope rope;  // rot_dim 0: no rotation
    const int32_t *starts;
    kvd_paged_cache cache;
};
cudaError_t launch_latent_append(const LatentAppendArgs &a, int x_dtype, cudaStream_t st);

// Attention over them: G is the number of query heads, c.head_dim the row's channels.
cudaError_t launch_latent_attn(const PagedAttnArgs &a, int rank, void *ws, cudaStream_t st);
size_t latent_attn_ws(int H, int rank, int max_new);

// Each cached token's weight, added up over the rows of its KV head.
struct MassArgs {
    PagedAttnArgs attn;  // out: unused; lse: read
    const float *mass;
    float *out;
    int64_t mass_stride, out_stride;  // from one (sequence, head) to the next
    float decay;
};
cudaError_t launch_mass(const MassArgs &a, cudaStream_t st);

struct EvictArgs {
    kvd_paged_cache c;  // v NULL: rows in k alone; k_scale and v_scale NULL: none
    int row_bytes;      // of k, and of v
    const float *mass;
    int64_t mass_stride;
    int keep, sink, recent;
    const int32_t *to;  // page table of the rows that stay
    int to_cols;
    int32_t *kept, *lens_out;
    float *mass_out;  // may be NULL
    int64_t mass_out_stride;
};
cudaError_t launch_evict(const EvictArgs &a, cudaStream_t st);

// Argument checks that the front ends share (paged_api.cu).
bool aligned(const void *p, size_t a);
kvd_status check_rows(const kvd_heads *h, int head_dim);
kvd_status check_rope(const kvd_rope *r, int head_dim, const float *qw, const float *kw, float eps);
kvd_status check_paged(const kvd_paged_cache *c);
kvd_status check_latent(const kvd_latent_cache *c);
// The latent cache as the kernels take it.
kvd_paged_cache latent_as_paged(const kvd_latent_cache &c);

}  // namespace kvd
