// paged_dev.cuh -- device helpers shared by the kernels of a ragged batch over
// a paged cache: the sequence of a token, and checked reads of the int32s that
// the caller keeps on the device.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace kvd {

// The sequence whose tokens [starts[b], starts[b + 1]) hold token t: the last
// b of [0, batch) with starts[b] <= t, by a search with 32 probes a step (one
// step up to 32 sequences, two up to 1024).  All lanes call it with the same
// t and get the same b; the caller checks t against starts[b] and starts[b + 1].
__device__ __forceinline__ int sequence_of(const int32_t *starts, int batch, int t, int lane) {
    int lo = 0, hi = batch;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + (lane + 1) * step;
        const bool below = at < hi && starts[at] <= t;
        const int n = __popc(__ballot_sync(0xffffffffu, below));
        lo += n * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

__device__ __forceinline__ int checked_len(const kvd_paged_cache &c, int b) {
    int l = c.seq_lens[b];
    if (l < 0 || l > c.len) {
        report_status(c.dev_status, KVD_ERR_INVALID);
        l = l < 0 ? 0 : c.len;
    }
    return l;
}

// The page of column j of sequence b, or -1 (and a report) for an entry
// outside the pool.
__device__ __forceinline__ int checked_page(const kvd_paged_cache &c, int b, int j) {
    const int p = c.page_table[static_cast<size_t>(b) * c.max_pages + j];
    if (p >= 0 && p < c.n_pages) return p;
    report_status(c.dev_status, KVD_ERR_INVALID);
    return -1;
}

// Two f32 as one word of f16 or bf16, each rounded to nearest even.
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    uint32_t w;
    if constexpr (BF16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
    return w;
}

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (BF16)
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    else
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

}  // namespace kvd
