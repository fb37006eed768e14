// paged_attn_int8.cu -- attention of a ragged batch's new tokens over a paged int8 cache.
//
//   out = sum_t softmax(scale q . k_t)_t v_t,   p - window < t <= p
//
// One warp per (token, query head): 32 keys at a time, a lane per key for the
// scores and a lane per channel pair for the values, with the running maximum
// and sum of the softmax.
#include "common.cuh"
#include "internal.h"
#include "paged.h"
#include "paged_dev.cuh"

namespace kvd {
namespace {

template <bool BF16, int DT>
__device__ __forceinline__ float2 cache2(const void *base, size_t at) {
    if constexpr (DT == KVD_INT8) {
        const char2 c = *reinterpret_cast<const char2 *>(static_cast<const int8_t *>(base) + at);
        return make_float2(static_cast<float>(c.x), static_cast<float>(c.y));
    } else {
        return unpack2<DT == KVD_BF16>(
            *reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(base) + at));
    }
}

template <bool BF16, int DT, int D>
__global__ void __launch_bounds__(128) attn_kernel(const __grid_constant__ PagedAttnArgs a) {
    __shared__ float2 qs[4][D / 2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x, h = blockIdx.y * 4 + warp;
    pdl_wait();
    pdl_launch_dependents();
    if (h >= a.H) return;
    const int b = sequence_of(a.starts, a.c.batch, t, lane);
    const int s0 = a.starts[b], s1 = a.starts[b + 1];
    if (t < s0 || t >= s1 || t - s0 >= a.max_new) {
        if (t < a.starts[a.c.batch]) report_status(a.c.dev_status, KVD_ERR_INVALID);
        return;
    }
    const long pos = static_cast<long>(checked_len(a.c, b)) - (s1 - t);
    if (pos < 0) report_status(a.c.dev_status, KVD_ERR_INVALID);
    const long first = a.window > 0 && pos - a.window + 1 > 0 ? pos - a.window + 1 : 0;
    const uint16_t *q = static_cast<const uint16_t *>(a.q) + t * a.q_stride + h * D;
    for (int i = lane; i < D / 2; i += 32)
        qs[warp][i] = unpack2<BF16>(reinterpret_cast<const uint32_t *>(q)[i]);
    __syncwarp();
    float m = -INFINITY, l = 0.0f;
    float2 acc[D / 64] = {};
    const int ps = a.c.page_size;
    for (long k0 = first / 32 * 32; k0 <= pos; k0 += 32) {
        const long kt = k0 + lane;
        int page = -1;
        size_t row = 0;
        if (kt >= first && kt <= pos) {
            const int j = static_cast<int>(kt / ps);
            page = checked_page(a.c, b, j);
            row = (static_cast<size_t>(page) * a.c.n_kv_heads + h / a.G) * ps + (kt - static_cast<long>(j) * ps);
        }
        float s = -INFINITY;
        if (page >= 0) {
            float dot = 0.0f;
            for (int i = 0; i < D / 2; ++i) {
                const float2 k = cache2<BF16, DT>(a.c.k, row * D + 2 * i);
                dot = fmaf(qs[warp][i].x, k.x, fmaf(qs[warp][i].y, k.y, dot));
            }
            if (DT == KVD_INT8) dot *= static_cast<const float *>(a.c.k_scale)[row];
            s = dot * a.scale_log2;
        }
        float mx = s;
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if (mx == -INFINITY) continue;
        const float mn = fmaxf(m, mx);
        const float alpha = exp2f(m - mn);
        float p = exp2f(s - mn);
        float sum = p;
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l = l * alpha + sum;
        m = mn;
        if (DT == KVD_INT8 && page >= 0) p *= static_cast<const float *>(a.c.v_scale)[row];
        for (int d = 0; d < D / 64; ++d) {
            acc[d].x *= alpha;
            acc[d].y *= alpha;
        }
        for (int u = 0; u < 32; ++u) {
            const int pg = __shfl_sync(0xffffffffu, page, u);
            const size_t r = __shfl_sync(0xffffffffu, row, u);
            const float pu = __shfl_sync(0xffffffffu, p, u);
            if (pg < 0) continue;
            for (int d = 0; d < D / 64; ++d) {
                const float2 v = cache2<BF16, DT>(a.c.v, r * D + 2 * (lane + 32 * d));
                acc[d].x = fmaf(pu, v.x, acc[d].x);
                acc[d].y = fmaf(pu, v.y, acc[d].y);
            }
        }
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    uint32_t *o = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) + t * a.out_stride + h * D);
    for (int d = 0; d < D / 64; ++d) o[lane + 32 * d] = pack2<BF16>(acc[d].x * inv, acc[d].y * inv);
}

template <bool BF16, int DT>
cudaError_t launch_d(const PagedAttnArgs &a, cudaStream_t st) {
    const dim3 grid(a.n_tokens, (a.H + 3) / 4);
    if (a.c.head_dim == 64)
        return launch_ex(attn_kernel<BF16, DT, 64>, grid, dim3(128), 0, st, true, a);
    return launch_ex(attn_kernel<BF16, DT, 128>, grid, dim3(128), 0, st, true, a);
}

}  // namespace

cudaError_t launch_paged_attn_simple(const PagedAttnArgs &a, cudaStream_t st) {
    return a.bf16 ? launch_d<true, KVD_INT8>(a, st) : launch_d<false, KVD_INT8>(a, st);
}

}  // namespace kvd
