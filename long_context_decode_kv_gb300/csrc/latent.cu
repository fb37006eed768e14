// latent.cu -- append to a paged cache of latent rows (kvd_latent_append).
//
//   row = [ c * w / sqrt(mean(c^2) + eps),  R(p) k_pe ]        q_out = R(p) q_pe
//
// One pass: each element is read once and written once.  A warp serves a token (several
// share one when a batch has few): the sines and cosines of its position are made once,
// turn the token's shared key part, and stay in registers for its 1 to 128 query heads,
// 4 heads at a time with 4 such groups in flight.  Angles as in rope.cu.
//
// Measured: 2 x 4095 tokens of 512 + 64 channels and 32 heads, f16, 20.3 us from HBM (4.2
// TB/s, 0.63 of what a copy reaches; 15.4 us where the L2 holds the inputs), bound by the
// warps' own chains (a token's place, its loads, the norm's sum) with DRAM at 31 % and the
// issue slots at 45 %; 64 tokens of 128 heads 4.2 us on the GPU.
#include "common.cuh"
#include "internal.h"
#include "paged.h"
#include "paged_dev.cuh"
#include "rope_dev.cuh"

namespace kvd {
namespace {

constexpr int kThreads = 128;
constexpr int kLanes = 8;              // that hold one head's rotated part (8 channels each)
constexpr int kHeadsAt = 32 / kLanes;  // heads a warp holds at once

// 8 neighbouring channels to a cache row of f16 or bf16.
__device__ __forceinline__ void store8(void *p, bool bf16, size_t at, const float2 (&x)[2][2]) {
    auto pack = [&](const float2 &v) {
        return bf16 ? pack2<true>(v.x, v.y) : pack2<false>(v.x, v.y);
    };
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + at) =
        make_uint4(pack(x[0][0]), pack(x[0][1]), pack(x[1][0]), pack(x[1][1]));
}

template <typename IN>
__global__ void __launch_bounds__(kThreads)
latent_append_kernel(const __grid_constant__ LatentAppendArgs a, int parts) {
    const int lane = threadIdx.x & 31;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    const int t = static_cast<int>(unit / parts), my_part = static_cast<int>(unit % parts);
    const int sub = lane / kLanes, col = lane % kLanes;
    const int W = a.rank + a.rope_dim;
    const bool bf16 = a.cache.dtype == KVD_BF16;
    pdl_wait();
    pdl_launch_dependents();
    if (t >= a.n_tokens) return;
    const TokenPlace at = place_of(a.cache, a.starts, a.n_tokens, t, lane);
    if (!at.some) return;
    const size_t row =
        (static_cast<size_t>(max(at.page, 0)) * a.cache.page_size + at.in_page) * W;

    // this lane's channels of a rotated part, and their cosines and sines
    const int2 ch = groups_of(a.rope, col);
    const bool on = 8 * col < a.rope_dim;
    float2 cs[2] = {splat(1.0f), splat(1.0f)}, sn[2] = {splat(0.0f), splat(0.0f)};
    if (8 * col < a.rope.rot_dim) {
        float c[4], s[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) angle_of(a.rope, at.pos, 4 * col + j, c[j], s[j]);
        cs[0] = make_float2(c[0], c[1]);
        cs[1] = make_float2(c[2], c[3]);
        sn[0] = make_float2(s[0], s[1]);
        sn[1] = make_float2(s[2], s[3]);
    }
    auto turn = [&](float2 (&x)[2][2]) {
        if (8 * col >= a.rope.rot_dim) return;
        if (a.rope.interleaved) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float2 c = cs[h], s = sn[h];
                float2 &p = x[h][0], &q = x[h][1];
                p = make_float2(fmaf(p.x, c.x, -p.y * s.x), fmaf(p.y, c.x, p.x * s.x));
                q = make_float2(fmaf(q.x, c.y, -q.y * s.y), fmaf(q.y, c.y, q.x * s.y));
            }
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float2 u0 = x[0][j], u1 = x[1][j];
                const float2 m = make_float2(-sn[j].x, -sn[j].y);
                x[0][j] = __ffma2_rn(u0, cs[j], __fmul2_rn(u1, m));
                x[1][j] = __ffma2_rn(u1, cs[j], __fmul2_rn(u0, sn[j]));
            }
        }
    };

    if (my_part == 0) {
        // the latent vector, 8 channels a lane and step
        const IN *src = static_cast<const IN *>(a.c.x) + t * a.c.stride;
        float2 x[2][2][2];
        Raw<IN> raw[2][2], key[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (8 * (lane + 32 * i) < a.rank) {
                raw[i][0].load(src + 8 * (lane + 32 * i));
                raw[i][1].load(src + 8 * (lane + 32 * i) + 4);
            }
        if (sub == 0 && on) {
            const IN *k = static_cast<const IN *>(a.k_pe.x) + t * a.k_pe.stride;
            key[0].load(k + ch.x);
            key[1].load(k + ch.y);
        }
        float2 sq = splat(0.0f);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (8 * (lane + 32 * i) >= a.rank) continue;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                raw[i][h].get(x[i][h]);
                sq = __ffma2_rn(x[i][h][0], x[i][h][0], sq);
                sq = __ffma2_rn(x[i][h][1], x[i][h][1], sq);
            }
        }
        if (a.c_weight) {
            float ss = sq.x + sq.y;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float2 rs = splat(rsqrtf(fmaf(ss, a.inv_rank, a.eps)));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (8 * (lane + 32 * i) >= a.rank) continue;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float2 w[2];
                    Raw<float> f;
                    f.load(a.c_weight + 8 * (lane + 32 * i) + 4 * h);
                    f.get(w);
                    x[i][h][0] = __fmul2_rn(x[i][h][0], __fmul2_rn(rs, w[0]));
                    x[i][h][1] = __fmul2_rn(x[i][h][1], __fmul2_rn(rs, w[1]));
                }
            }
        }
        if (at.page >= 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (8 * (lane + 32 * i) < a.rank)
                    store8(a.cache.k, bf16, row + 8 * (lane + 32 * i), x[i]);
            if (sub == 0 && on) {
                float2 y[2][2];
                key[0].get(y[0]);
                key[1].get(y[1]);
                turn(y);
                const int type = bf16 ? KVD_X_BF16 : KVD_X_F16;
                store4(a.cache.k, type, row + a.rank + ch.x, y[0]);
                store4(a.cache.k, type, row + a.rank + ch.y, y[1]);
            }
        }
    }

    // the queries' parts: groups of kHeadsAt heads, every parts-th this warp's
    const int groups = (a.q.n_heads + kHeadsAt - 1) / kHeadsAt;
    const IN *src = static_cast<const IN *>(a.q.x) + t * a.q.stride;
    constexpr int U = 4;
    Raw<IN> raw[U][2];
    auto load = [&](int u, int g) {
        const int h = g * kHeadsAt + sub;
        if (on && g < groups && h < a.q.n_heads) {
            raw[u][0].load(src + h * a.q_head + ch.x);
            raw[u][1].load(src + h * a.q_head + ch.y);
        }
    };
#pragma unroll
    for (int u = 0; u < U; ++u) load(u, my_part + u * parts);
    for (int g = my_part; g < groups; g += U * parts) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at_g = g + u * parts, h = at_g * kHeadsAt + sub;
            float2 y[2][2];
            const bool ok = on && at_g < groups && h < a.q.n_heads;
            if (ok) {
                raw[u][0].get(y[0]);
                raw[u][1].get(y[1]);
            }
            load(u, at_g + U * parts);
            if (ok) {
                turn(y);
                const size_t to = static_cast<size_t>(t * a.q_out.stride + h * a.q_out_head);
                store4(a.q_out.x, a.q_out.dtype, to + ch.x, y[0]);
                store4(a.q_out.x, a.q_out.dtype, to + ch.y, y[1]);
            }
        }
    }
}

template <typename IN>
cudaError_t launch(const LatentAppendArgs &a, cudaStream_t st) {
    // warps a token: one, or as many as give every SM 16 warps
    const int most = 1 + (a.q.n_heads + kHeadsAt - 1) / kHeadsAt;
    const int64_t want = (16ll * device_sm_count() + a.n_tokens - 1) / a.n_tokens;
    const int parts = want < most ? static_cast<int>(want) : most;
    const int64_t units = static_cast<int64_t>(a.n_tokens) * parts;
    constexpr int kWarps = kThreads / 32;
    return launch_ex(latent_append_kernel<IN>,
                     dim3(static_cast<unsigned>((units + kWarps - 1) / kWarps)), dim3(kThreads), 0,
                     st, true, a, parts);
}

}  // namespace

cudaError_t launch_latent_append(const LatentAppendArgs &a, int x_dtype, cudaStream_t st) {
    if (x_dtype == KVD_X_F16) return launch<__half>(a, st);
    if (x_dtype == KVD_X_BF16) return launch<__nv_bfloat16>(a, st);
    return launch<float>(a, st);
}

}  // namespace kvd
