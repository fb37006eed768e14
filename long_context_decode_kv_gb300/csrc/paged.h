// paged.h -- launchers of the norm/rotation, paged append and paged attention
// kernels (rope.cu, paged_attn.cu, paged_decode.cu) for their C-ABI front end (paged_api.cu).
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

}  // namespace kvd
