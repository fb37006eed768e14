// paged_attn_dev.cuh -- what the two attention kernels over a paged cache share:
// their arguments, the sequences' checked lengths, the waits between warp roles,
// the reading of int8 codes, and the tensor maps of the launch.
#pragma once

#include <cuda.h>

#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "paged.h"
#include "paged_dev.cuh"
#include "tcgen05.cuh"

namespace kvd {

constexpr int kTile = 128;  // keys a tile

struct AttnArgs {  // of a launch
    kvd_paged_cache c;
    uint16_t *out;
    int64_t out_stride;
    int G, n_tokens, max_new, window;
    const int32_t *starts;
    float scale_log2;
    int box;            // cache rows a TMA box: the largest of 16..128 that divides a page
    int dead_row;       // a cache row outside the pool
    int min_tiles;      // least key tiles a CTA takes (row tiles: with what an item costs)
    float *lse;         // [n_tokens][n_kv_heads * G] or NULL
};

// A row's statistic from the reference m (base 2) and the sum l of its weights 2^(logit - m).
// References stand below the row's maximum, so l is above 16 where it is not 0: far from 1,
// where the fast logarithm is good to 2 units in the last place.  That is an absolute error, as
// m and log2(l) may cancel: 2^-19 for l below 2^16 (2^-17 for any), times ln 2; the sum, the
// product and the constant add 2.5 * 2^-24 of |lse|.  As a factor exp(-lse) of a weight it is the
// same relative error: 2^-19.5, and with the weight's own use of lse 2^-22 of |lse|.
__device__ __forceinline__ float lse_of(float m, float l) {
    return l > 0.0f || l != l ? (m + __log2f(l)) * 0.69314718056f : -INFINITY;
}
// Where it stands: token t, query head h of KV head `head`.
__device__ __forceinline__ float *lse_at(const AttnArgs &a, int t, int head, int h) {
    return a.lse + static_cast<int64_t>(t) * (a.c.n_kv_heads * a.G) + head * a.G + h;
}

// mbar_wait for the waits between the roles, in few instructions: the roles' hot
// lines have to fit the instruction cache together, and a wait mostly ends in its
// first try.  Warps call it whole, and all lanes get the same answer.  limit_ns < 2^32.
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, volatile int *abort,
                                         uint32_t limit_ns = static_cast<uint32_t>(kWaitLimitNs)) {
    uint32_t n = 0, t0 = 0;
#pragma unroll 1
    while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) {
        if ((++n & 63u) == 0) {
            const uint32_t t = static_cast<uint32_t>(global_timer_ns());
            if (n == 64) t0 = t;
            if (__any_sync(0xffffffffu, *abort || t - t0 > limit_ns)) return false;
        }
    }
    return true;
}

// The wait of lanes with a barrier each: those that take part (`mine`) do f() as soon as
// their own barrier's phase has completed, whichever comes first.
template <typename F>
__device__ __forceinline__ bool each_when(bool mine, uint64_t *bar, uint32_t parity,
                                          volatile int *abort, F f,
                                          uint32_t limit_ns = static_cast<uint32_t>(kWaitLimitNs)) {
    uint32_t n = 0, t0 = 0;
#pragma unroll 1
    while (__any_sync(0xffffffffu, mine)) {
        if (mine && mbar_try_wait(bar, parity)) {
            f();
            mine = false;
        }
        if ((++n & 63u) == 0) {
            const uint32_t t = static_cast<uint32_t>(global_timer_ns());
            if (n == 64) t0 = t;
            if (__any_sync(0xffffffffu, *abort || t - t0 > limit_ns)) return false;
        }
    }
    return true;
}

// ------------------------------------------------------------ sequences ---
struct Seq {
    int s0, n, len;  // first token, new tokens (at most max_new), length
    int first;       // position of the first new token
};

__device__ __forceinline__ Seq seq_of(const AttnArgs &a, int b, bool report) {
    const int r0 = a.starts[b], r1 = a.starts[b + 1];
    int len = a.c.seq_lens[b];
    const int s0 = min(max(r0, 0), a.n_tokens);
    const int s1 = min(max(r1, s0), a.n_tokens);
    const int l = min(max(len, 0), a.c.len);
    Seq s{s0, min(s1 - s0, a.max_new), l, l - (s1 - s0)};
    if (report && (r0 != s0 || r1 != s1 || l != len || s1 - s0 > a.max_new || s.first < 0))
        report_status(a.c.dev_status, KVD_ERR_INVALID);
    return s;
}

// int8: weights are stored times their values' scales, in units of 2^exp, and O is
// counted in the same units.  The exponent follows the tiles' largest scales in both
// directions (O is scaled where it changes), so that a tile with one far larger scale
// takes f16's range from its own keys alone and not from all that follow it.
struct ScaleUnit {
    int exp, peak;  // the peak of the run of tiles so far
    // The bits of a tile's largest finite scale (0: none but zeros).  `room`: how many
    // places scales may pass the unit.  It falls where they are more than 5 below (the
    // weights' lift stands against those 5; a change costs a pass over O, so scales that
    // merely vary should cause none), and to at most 60 below the peak, from where O in
    // smaller units could overflow f32.
    __device__ __forceinline__ void take(uint32_t top, bool first, int room) {
        const int e = min(max(static_cast<int>(top >> 23) - 126, -100), 100);
        if (first)
            exp = peak = e;
        else if (e > exp + room)
            exp = e;
        else if (e < exp - 5 && top != 0)
            exp = max(e, peak - 60);
        peak = max(peak, exp);
    }
};

// Four int8 codes as two words of f16 or bf16, exactly.  f16: code + 128 in the
// low bits of 1024 + x, less 1152.  bf16: 128 + (code's low 7 bits), less 128 or,
// for a negative code, 256.
template <bool BF16>
__device__ __forceinline__ void codes_to(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if constexpr (BF16) {
        const uint32_t t0 = __byte_perm(w, 0, 0x4140), t1 = __byte_perm(w, 0, 0x4342);
        auto sub = [](uint32_t t) {
            const uint32_t x = (t & 0x007f007fu) | 0x43004300u, y = (t & 0x00800080u) | 0x43004300u;
            const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&x),
                                             *reinterpret_cast<const __nv_bfloat162 *>(&y));
            return *reinterpret_cast<const uint32_t *>(&d);
        };
        lo = sub(t0);
        hi = sub(t1);
    } else {
        const uint32_t u = w ^ 0x80808080u;
        const uint32_t k1152 = 0x64806480u;
        auto sub = [&](uint32_t x) {
            const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&x),
                                      *reinterpret_cast<const __half2 *>(&k1152));
            return *reinterpret_cast<const uint32_t *>(&d);
        };
        lo = sub(__byte_perm(u, 0x64646464u, 0x4140));
        hi = sub(__byte_perm(u, 0x64646464u, 0x4342));
    }
}

// ---------------------------------------------------------------- launch ---
using EncodeTiled = decltype(&cuTensorMapEncodeTiled);

// The driver's encoder of tensor maps, asked of the runtime once.
inline EncodeTiled encoder() {
    static std::atomic<void *> fn{nullptr};
    void *p = fn.load(std::memory_order_relaxed);
    if (!p) {
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            return nullptr;
        fn.store(p, std::memory_order_relaxed);
    }
    return reinterpret_cast<EncodeTiled>(p);
}

inline bool make_map(CUtensorMap *m, int kv_dtype, const void *base, int rank,
                     const cuuint64_t *dims, const cuuint64_t *strides, const cuuint32_t *box,
                     CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
    const EncodeTiled enc = encoder();
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    const CUtensorMapDataType type = kv_dtype == KVD_INT8   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : kv_dtype == KVD_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                            : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    return enc && enc(m, type, rank, const_cast<void *>(base), dims, strides, box, ones,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A launch's arguments and its tensor maps of q (boxes of q_tokens tokens of one
// KV head), k and v (boxes of a page's rows).
inline bool fill_launch(const PagedAttnArgs &p, int q_tokens, CUtensorMapSwizzle k_swizzle,
                        CUtensorMapSwizzle v_swizzle, AttnArgs &a, CUtensorMap &q_map,
                        CUtensorMap &k_map, CUtensorMap &v_map) {
    const kvd_paged_cache &c = p.c;
    const bool i8 = c.dtype == KVD_INT8;
    a.c = c;
    a.out = static_cast<uint16_t *>(p.out);
    a.out_stride = p.out_stride;
    a.G = p.G;
    a.n_tokens = p.n_tokens;
    a.max_new = p.max_new;
    a.window = p.window;
    a.starts = p.starts;
    a.scale_log2 = p.scale_log2;
    a.lse = p.lse;
    a.box = 16;
    while (a.box < kTile && c.page_size % (2 * a.box) == 0) a.box *= 2;
    const int64_t rows = static_cast<int64_t>(c.n_pages) * c.n_kv_heads * c.page_size;
    a.dead_row = static_cast<int>(rows);
    const cuuint64_t D = static_cast<cuuint64_t>(c.head_dim);
    const cuuint64_t qd[4] = {D, static_cast<cuuint64_t>(p.G),
                              static_cast<cuuint64_t>(c.n_kv_heads),
                              static_cast<cuuint64_t>(p.n_tokens)};
    const cuuint64_t qs[3] = {D * 2, D * 2 * p.G, static_cast<cuuint64_t>(p.q_stride) * 2};
    const cuuint32_t qb[4] = {64, static_cast<cuuint32_t>(p.G), 1,
                              static_cast<cuuint32_t>(q_tokens)};
    const cuuint64_t kd[2] = {D, static_cast<cuuint64_t>(rows)};
    const cuuint64_t ks[1] = {D * (i8 ? 1 : 2)};
    const cuuint32_t kb[2] = {i8 ? static_cast<cuuint32_t>(D) : 64, static_cast<cuuint32_t>(a.box)};
    return make_map(&q_map, p.bf16 ? KVD_BF16 : KVD_F16, p.q, 4, qd, qs, qb) &&
           make_map(&k_map, c.dtype, c.k, 2, kd, ks, kb, k_swizzle) &&
           make_map(&v_map, c.dtype, c.v, 2, kd, ks, kb, v_swizzle);
}

}  // namespace kvd
