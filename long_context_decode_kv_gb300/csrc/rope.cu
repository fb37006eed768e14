// rope.cu -- per-head RMS norm and position rotation of queries and keys, alone
// (kvd_qk_norm_rope) or with the append to a paged cache (kvd_paged_append).
//
//   y = R(p) (x * w / sqrt(mean(x^2) + eps))
//   R(p) turns channel pair i of the first rot_dim channels by p * f_i.
//
// Each element is read once and written once, and the least it can take is HBM's time
// for that.  What has to be kept down is the work on each: a lane holds the two channel groups that turn into
// each other (4 channels of the lower and 4 of the upper half; 8 neighbours when
// pairs are interleaved), so no lane needs another's values but for the sum of
// the norm, and two channels share an instruction (FFMA2).  A warp serves one
// token (several share one when a batch has few): the sines and cosines of its
// channels and the norms' weights are made once, stay in registers, and serve the
// token's 10 to 100 heads.  A row of head_dim channels is held by the fewest lanes
// that take 8 channels each (16 at 128), with U rows a lane in flight.
//
// The angle: the frequency is a 64-bit fraction of a turn per position, so the
// product with the position, modulo 2^64, is the angle's fraction of a turn with
// an error below position * 2^-64; its upper 32 bits go to sincospi.  In f32 the
// product alone is off by 2^-24 of itself: 0.06 radians at position 1,000,000.
//
// Measured: 8192 tokens of 32 + 8 heads, bf16, normed and rotated 32.8 us (5.1 TB/s,
// 0.75 of what a copy reaches); 8190 tokens of 32 + 8 + 8 appended to pages 45 us
// (4.4 TB/s), to int8 pages 58.  Neither HBM (45 and 42 % of its cycles in a single cold
// launch) nor the issue slots (56 and 48 %) hold these alone: an SM has 26 and 20 warps
// at a time, and each waits on the reads and the fixed latencies of its own chain.  A
// few tokens take a launch and its host call, 8.7 us.
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "paged.h"
#include "paged_dev.cuh"
#include "rope_dev.cuh"

namespace kvd {
namespace {

constexpr int kThreads = 128;

// LPR lanes hold one row, lane l chunks l, l + LPR, .. (VPL of them).
template <typename IN, int LPR, int VPL, int U, bool PAGED>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a,
                                                        int parts) {
    const int lane = threadIdx.x & 31;
    const int unit = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int t = unit / parts, my_part = unit % parts;
    constexpr int kRows = 32 / LPR;  // a warp holds at once: a group
    const int sub = lane / LPR, col = lane % LPR;
    const int chunks = a.head_dim / 8;
    pdl_wait();
    pdl_launch_dependents();
    if (t >= a.n_tokens) return;

    int2 ch[VPL];
    bool on[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        ch[i] = groups_of(a.rope, col + i * LPR);
        on[i] = col + i * LPR < chunks;
    }

    // the token's position, and with a cache the place of its rows
    long pos = 0;
    size_t row0 = 0;  // cache row of KV head 0
    bool store_kv = false;
    if constexpr (PAGED) {
        const TokenPlace at = place_of(a.cache, a.starts, a.n_tokens, t, lane);
        if (!at.some) return;
        pos = at.pos;
        store_kv = at.page >= 0;
        if (store_kv)
            row0 = static_cast<size_t>(at.page) * a.cache.n_kv_heads * a.cache.page_size + at.in_page;
    } else if (a.rope.rot_dim) {
        pos = a.positions[t];
    }

    // The lane's cosines and sines times mscale: of the 4 pairs of a chunk, as
    // (pair 0, pair 1), (pair 2, pair 3).  Channels that are not rotated: (1, 0).
    float2 cs[VPL][2], sn[VPL][2];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        float c[4] = {1.0f, 1.0f, 1.0f, 1.0f}, s[4] = {};
        if (8 * (col + i * LPR) < a.rope.rot_dim) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                angle_of(a.rope, pos, 4 * (col + i * LPR) + j, c[j], s[j]);
        }
        cs[i][0] = make_float2(c[0], c[1]);
        cs[i][1] = make_float2(c[2], c[3]);
        sn[i][0] = make_float2(s[0], s[1]);
        sn[i][1] = make_float2(s[2], s[3]);
    }

    // The rows of q (PART 0), k (1) or v (2), whose groups of kRows are numbered
    // on from group g0: every parts-th is this warp's.
    auto run = [&](auto part_tag, const RowsIn &in, int g0, const float *weight) {
        constexpr int PART = decltype(part_tag)::value;
        const int ng = (in.n_heads + kRows - 1) / kRows;
        int g = g0 <= my_part ? my_part - g0
                              : (parts - (g0 - my_part) % parts) % parts;  // first of ours
        if (g >= ng) return;
        const IN *src = static_cast<const IN *>(in.x) + t * in.stride;
        Raw<IN> raw[U][VPL][2];
        auto load = [&](int u, int at) {
            const int r = at * kRows + sub;
            if (at < ng && r < in.n_heads)
#pragma unroll
                for (int i = 0; i < VPL; ++i)
                    if (on[i]) {
                        raw[u][i][0].load(src + r * a.head_dim + ch[i].x);
                        raw[u][i][1].load(src + r * a.head_dim + ch[i].y);
                    }
        };
#pragma unroll
        for (int u = 0; u < U; ++u) load(u, g + u * parts);
        float2 w[VPL][2][2];
        if (PART < 2 && weight)
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (on[i]) {
                    Raw<float> f;
                    f.load(weight + ch[i].x);
                    f.get(w[i][0]);
                    f.load(weight + ch[i].y);
                    f.get(w[i][1]);
                }
        for (; g < ng; g += U * parts) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (g + u * parts >= ng) break;  // the same for the whole warp
                const int r = (g + u * parts) * kRows + sub;
                const bool ok = r < in.n_heads;
                float2 x[VPL][2][2];
#pragma unroll
                for (int i = 0; i < VPL; ++i) {
                    raw[u][i][0].get(x[i][0]);
                    raw[u][i][1].get(x[i][1]);
                    if (!ok || !on[i])
                        x[i][0][0] = x[i][0][1] = x[i][1][0] = x[i][1][1] = splat(0.0f);
                }
                load(u, g + (u + U) * parts);
                if (PART < 2 && weight) {
                    float2 sq = splat(0.0f);
#pragma unroll
                    for (int i = 0; i < VPL; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            sq = __ffma2_rn(x[i][h][0], x[i][h][0], sq);
                            sq = __ffma2_rn(x[i][h][1], x[i][h][1], sq);
                        }
                    float ss = sq.x + sq.y;
#pragma unroll
                    for (int o = LPR / 2; o > 0; o >>= 1)
                        ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    const float2 rs = splat(rsqrtf(fmaf(ss, a.inv_dim, a.eps)));
#pragma unroll
                    for (int i = 0; i < VPL; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            x[i][h][0] = __fmul2_rn(x[i][h][0], __fmul2_rn(rs, w[i][h][0]));
                            x[i][h][1] = __fmul2_rn(x[i][h][1], __fmul2_rn(rs, w[i][h][1]));
                        }
                }
                if (PART < 2 && a.rope.rot_dim) {
                    if (a.rope.interleaved) {
#pragma unroll
                        for (int i = 0; i < VPL; ++i)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const float2 c = cs[i][h], s = sn[i][h];
                                float2 &p = x[i][h][0], &q = x[i][h][1];
                                p = make_float2(fmaf(p.x, c.x, -p.y * s.x),
                                                fmaf(p.y, c.x, p.x * s.x));
                                q = make_float2(fmaf(q.x, c.y, -q.y * s.y),
                                                fmaf(q.y, c.y, q.x * s.y));
                            }
                    } else {
#pragma unroll
                        for (int i = 0; i < VPL; ++i)
                            if (8 * (col + i * LPR) < a.rope.rot_dim)
#pragma unroll
                                for (int j = 0; j < 2; ++j) {
                                    const float2 u0 = x[i][0][j], u1 = x[i][1][j];
                                    const float2 c = cs[i][j], s = sn[i][j];
                                    const float2 m = make_float2(-s.x, -s.y);
                                    x[i][0][j] = __ffma2_rn(u0, c, __fmul2_rn(u1, m));
                                    x[i][1][j] = __ffma2_rn(u1, c, __fmul2_rn(u0, s));
                                }
                    }
                }
                if constexpr (PART == 0 || !PAGED) {
                    const RowsOut &o = PART == 0 ? a.q_out : a.k_out;
                    const size_t at = static_cast<size_t>(t * o.stride) +
                                      static_cast<size_t>(r) * a.head_dim;
#pragma unroll
                    for (int i = 0; i < VPL; ++i)
                        if (ok && on[i]) {
                            store4(o.x, o.dtype, at + ch[i].x, x[i][0]);
                            store4(o.x, o.dtype, at + ch[i].y, x[i][1]);
                        }
                } else {
                    static_assert(VPL == 1 || !PAGED, "paged head dims fit one chunk a lane");
                    const size_t row = row0 + static_cast<size_t>(r) * a.cache.page_size;
                    void *dst = PART == 1 ? a.cache.k : a.cache.v;
                    const bool kv = ok && store_kv && on[0];
                    if (a.cache.dtype == KVD_INT8) {
                        float m = 0.0f;
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                m = fmaxf(m, fmaxf(fabsf(x[0][h][j].x), fabsf(x[0][h][j].y)));
#pragma unroll
                        for (int o = LPR / 2; o > 0; o >>= 1)
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                        const float s = __fdiv_rn(m, 127.0f);
                        auto code = [&](float v) -> uint32_t {
                            if (s == 0.0f) return 0u;
                            const int c = __float2int_rn(__fdiv_rn(v, s));
                            return static_cast<uint32_t>(max(-127, min(127, c))) & 0xffu;
                        };
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t w4 = code(x[0][h][0].x) | code(x[0][h][0].y) << 8 |
                                                code(x[0][h][1].x) << 16 | code(x[0][h][1].y) << 24;
                            if (kv)
                                *reinterpret_cast<uint32_t *>(static_cast<int8_t *>(dst) +
                                                              row * a.head_dim +
                                                              (h ? ch[0].y : ch[0].x)) = w4;
                        }
                        if (kv && col == 0)
                            static_cast<float *>(PART == 1 ? a.cache.k_scale
                                                           : a.cache.v_scale)[row] = s;
                    } else if (kv) {
                        const int type = a.cache.dtype == KVD_BF16 ? KVD_X_BF16 : KVD_X_F16;
                        store4(dst, type, row * a.head_dim + ch[0].x, x[0][0]);
                        store4(dst, type, row * a.head_dim + ch[0].y, x[0][1]);
                    }
                }
            }
        }
    };
    const int gq = (a.q.n_heads + kRows - 1) / kRows, gk = (a.k.n_heads + kRows - 1) / kRows;
    if (a.q.n_heads) run(std::integral_constant<int, 0>(), a.q, 0, a.q_weight);
    if (a.k.n_heads) run(std::integral_constant<int, 1>(), a.k, gq, a.k_weight);
    if constexpr (PAGED) run(std::integral_constant<int, 2>(), a.v, gq + gk, nullptr);
}

template <typename IN, int LPR, int VPL, int U, bool PAGED>
cudaError_t launch(const RopeArgs &a, cudaStream_t st) {
    constexpr int kRows = 32 / LPR;
    // Warps a token: one, or as many as give every SM 16 warps (a few tokens' heads
    // would otherwise follow one another in one warp)
    const int most = (a.q.n_heads + kRows - 1) / kRows + (a.k.n_heads + kRows - 1) / kRows +
                     (a.v.n_heads + kRows - 1) / kRows;
    const int64_t want = (16ll * device_sm_count() + a.n_tokens - 1) / a.n_tokens;
    const int parts = want < most ? static_cast<int>(want) : most;
    const int64_t units = static_cast<int64_t>(a.n_tokens) * parts;
    constexpr int kWarps = kThreads / 32;
    return launch_ex(rope_kernel<IN, LPR, VPL, U, PAGED>,
                     dim3(static_cast<unsigned>((units + kWarps - 1) / kWarps)), dim3(kThreads), 0,
                     st, true, a, parts);
}

template <typename IN>
cudaError_t launch_in(const RopeArgs &a, cudaStream_t st) {
    const bool paged = a.cache.page_table != nullptr;
    if (a.head_dim <= 64)
        return paged ? launch<IN, 8, 1, 4, true>(a, st) : launch<IN, 8, 1, 4, false>(a, st);
    if (a.head_dim <= 128)
        return paged ? launch<IN, 16, 1, 4, true>(a, st) : launch<IN, 16, 1, 4, false>(a, st);
    if (a.head_dim <= 256) return launch<IN, 32, 1, 2, false>(a, st);
    return launch<IN, 32, 4, 1, false>(a, st);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, int x_dtype, cudaStream_t st) {
    if (x_dtype == KVD_X_F16) return launch_in<__half>(a, st);
    if (x_dtype == KVD_X_BF16) return launch_in<__nv_bfloat16>(a, st);
    return launch_in<float>(a, st);
}

}  // namespace kvd
