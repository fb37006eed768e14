// rope_dev.cuh -- device helpers of the kernels that norm, rotate and append rows: four
// channels at a time in and out, which channels turn into each other, and the angles.
#pragma once

#include <type_traits>

#include "paged_dev.cuh"

namespace kvd {

// 4 channels as loaded.
template <typename T>
struct Raw {
    uint2 w;
    __device__ __forceinline__ void load(const void *p) { w = *static_cast<const uint2 *>(p); }
    __device__ __forceinline__ void get(float2 (&x)[2]) const {
        constexpr bool kBf16 = !std::is_same<T, __half>::value;
        x[0] = unpack2<kBf16>(w.x);
        x[1] = unpack2<kBf16>(w.y);
    }
};
template <>
struct Raw<float> {
    float4 w;
    __device__ __forceinline__ void load(const void *p) { w = *static_cast<const float4 *>(p); }
    __device__ __forceinline__ void get(float2 (&x)[2]) const {
        x[0] = make_float2(w.x, w.y);
        x[1] = make_float2(w.z, w.w);
    }
};

// 4 channels to element `at` of an array of the given type.
__device__ __forceinline__ void store4(void *p, int dtype, size_t at, const float2 (&x)[2]) {
    if (dtype == KVD_X_F32)
        *reinterpret_cast<float4 *>(static_cast<float *>(p) + at) =
            make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
    else
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p) + at) =
            dtype == KVD_X_BF16
                ? make_uint2(pack2<true>(x[0].x, x[0].y), pack2<true>(x[1].x, x[1].y))
                : make_uint2(pack2<false>(x[0].x, x[0].y), pack2<false>(x[1].x, x[1].y));
}

__device__ __forceinline__ float2 splat(float x) { return make_float2(x, x); }

// The first channels of the two groups of 4 that chunk c of a row holds.
__device__ __forceinline__ int2 groups_of(const kvd_rope &r, int c) {
    if (!r.interleaved && c < r.rot_dim / 8) return make_int2(4 * c, r.rot_dim / 2 + 4 * c);
    return make_int2(8 * c, 8 * c + 4);  // no pair apart: neighbours
}

// Cosine and sine of pair i at position pos, times mscale: the frequency is a 64-bit
// fraction of a turn, so the product modulo 2^64 is the angle's, and its signed upper
// half counts half turns in [-1, 1).
__device__ __forceinline__ void angle_of(const kvd_rope &r, long pos, int i, float &c, float &s) {
    const uint64_t frac = static_cast<uint64_t>(pos) * r.freqs[i];
    const float x = static_cast<float>(static_cast<int32_t>(frac >> 32)) * 0x1p-31f;
    sincospif(x, &s, &c);
    c *= r.mscale;
    s *= r.mscale;
}

}  // namespace kvd
