// rope.cu -- per-head RMS norm and position rotation of queries and keys, alone
// (kvd_qk_norm_rope) or with the append to a paged cache (kvd_paged_append).
//
//   y = R(p) (x * w / sqrt(mean(x^2) + eps))
//   R(p) turns channel pair i of the first rot_dim channels by p * f_i.
//
// Bound by HBM: each element is read once and written once.  A warp serves one
// token (several share one when a batch has few), so the sines and cosines of a
// lane's channels and the norms' weights are made once, stay in registers, and
// serve the token's 10 to 100 heads; no lane waits for another warp.  A row of
// head_dim channels is held by the fewest lanes that take 8 channels each (16
// lanes at 128), so a warp moves 512 contiguous bytes of f16 an instruction, with
// U such loads in flight.
//
// The angle: the frequency is a 64-bit fraction of a turn per position, so the
// product with the position, modulo 2^64, is the angle's fraction of a turn with
// an error below position * 2^-64; its upper 32 bits go to sincospi.  In f32 the
// product alone is off by 2^-24 of itself: 0.06 radians at position 1,000,000.
#include "common.cuh"
#include "internal.h"
#include "paged.h"
#include "paged_dev.cuh"

namespace kvd {
namespace {

constexpr int kThreads = 128;

template <typename T>
struct Raw {  // 8 channels as loaded: f16 or bf16
    uint4 w;
    __device__ __forceinline__ void load(const void *p) { w = *static_cast<const uint4 *>(p); }
    __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = unpack2<sizeof(T) == 2 && !std::is_same<T, __half>::value>(u[j]);
            x[2 * j] = f.x;
            x[2 * j + 1] = f.y;
        }
    }
};
template <>
struct Raw<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const void *p) {
        a = static_cast<const float4 *>(p)[0];
        b = static_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
};

// 8 channels to element `at` of an array of the given type.
__device__ __forceinline__ void store8(void *p, int dtype, size_t at, const float (&x)[8]) {
    if (dtype == KVD_X_F32) {
        float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(p) + at);
        o[0] = make_float4(x[0], x[1], x[2], x[3]);
        o[1] = make_float4(x[4], x[5], x[6], x[7]);
        return;
    }
    uint4 w;
    if (dtype == KVD_X_BF16)
        w = make_uint4(pack2<true>(x[0], x[1]), pack2<true>(x[2], x[3]), pack2<true>(x[4], x[5]),
                       pack2<true>(x[6], x[7]));
    else
        w = make_uint4(pack2<false>(x[0], x[1]), pack2<false>(x[2], x[3]),
                       pack2<false>(x[4], x[5]), pack2<false>(x[6], x[7]));
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + at) = w;
}

// LPR lanes hold one row, lane l chunks l, l + LPR, .. (8 channels each, VPL of
// them); U rows a lane group are in flight.
template <typename IN, int LPR, int VPL, int U, bool PAGED>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a,
                                                        int parts) {
    const int lane = threadIdx.x & 31;
    const int unit = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int t = unit / parts;
    constexpr int kRows = 32 / LPR;  // a warp holds at once
    const int sub = lane / LPR, col = lane % LPR;
    const int nrows = a.q.n_heads + a.k.n_heads + a.v.n_heads;
    const int chunks = a.head_dim / 8;
    const int step = parts * kRows, r0 = unit % parts * kRows;
    pdl_wait();
    pdl_launch_dependents();
    if (t >= a.n_tokens) return;

    Raw<IN> raw[U][VPL];
    auto load = [&](int u, int r) {  // row r into raw[u]
        const bool ok = r < nrows;
        const RowsIn *in = &a.q;
        if (r >= a.q.n_heads) {
            r -= a.q.n_heads;
            in = &a.k;
            if (r >= a.k.n_heads) {
                r -= a.k.n_heads;
                in = &a.v;
            }
        }
        const IN *src = static_cast<const IN *>(in->x) + t * in->stride +
                        static_cast<int64_t>(r) * a.head_dim;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int c = col + i * LPR;
            if (ok && c < chunks)
                raw[u][i].load(src + 8 * c);
            else
                raw[u][i].zero();
        }
    };
#pragma unroll
    for (int u = 0; u < U; ++u) load(u, r0 + u * step + sub);

    // the token's position, and with a cache the place of its rows
    long pos = 0;
    size_t row0 = 0;  // cache row of KV head 0
    bool store_kv = false;
    if constexpr (PAGED) {
        const int b = sequence_of(a.starts, a.cache.batch, t, lane);
        const int s0 = a.starts[b], s1 = a.starts[b + 1], end = a.starts[a.cache.batch];
        if (t < s0 || t >= s1) {
            // behind the last sequence, or starts that are not in order
            if (t < end && lane == 0) report_status(a.cache.dev_status, KVD_ERR_INVALID);
            return;
        }
        pos = static_cast<long>(checked_len(a.cache, b)) - (s1 - t);
        if (pos >= 0) {
            const int ps = a.cache.page_size;
            const int j = static_cast<int>(pos) / ps;
            const int page = checked_page(a.cache, b, j);
            store_kv = page >= 0;
            row0 = static_cast<size_t>(page) * a.cache.n_kv_heads * ps + (pos - j * ps);
        } else if (lane == 0) {
            report_status(a.cache.dev_status, KVD_ERR_INVALID);
        }
    } else if (a.rope.rot_dim) {
        pos = a.positions[t];
    }

    // (cos, sin) * mscale of this lane's channels: for pairs (i, i + rot_dim / 2)
    // of all 8 of a chunk, with the sign of the other channel's share; interleaved,
    // of its 4 pairs.  Channels that are not rotated: (1, 0).
    const int half = a.rope.rot_dim / 2;
    float cs[VPL][8], sn[VPL][8];
    if (half) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int ch = 8 * (col + i * LPR);
            const bool turns = ch < 2 * half;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                cs[i][j] = 1.0f;
                sn[i][j] = 0.0f;
                if (!turns || (a.rope.interleaved && j >= 4)) continue;
                const int pair = a.rope.interleaved ? ch / 2 + j : ch < half ? ch + j : ch - half + j;
                const uint64_t frac = static_cast<uint64_t>(pos) * a.rope.freqs[pair];
                // signed upper half: half turns in [-1, 1)
                const float x = static_cast<float>(static_cast<int32_t>(frac >> 32)) * 0x1p-31f;
                float s, c;
                sincospif(x, &s, &c);
                cs[i][j] = c * a.rope.mscale;
                sn[i][j] = (a.rope.interleaved || ch >= half ? s : -s) * a.rope.mscale;
            }
        }
    }
    float wq[VPL][8] = {}, wk[VPL][8] = {};
    const bool norms = a.q_weight || a.k_weight;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int c = col + i * LPR;
        Raw<float> w;
        if (a.q_weight && c < chunks) {
            w.load(a.q_weight + 8 * c);
            w.get(wq[i]);
        }
        if (a.k_weight && c < chunks) {
            w.load(a.k_weight + 8 * c);
            w.get(wk[i]);
        }
    }

    for (int base = r0; base < nrows; base += U * step) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (base + u * step >= nrows) break;  // the same for the whole warp
            int r = base + u * step + sub;
            const bool ok = r < nrows;
            int part = 0;
            if (r >= a.q.n_heads) {
                r -= a.q.n_heads;
                part = 1;
                if (r >= a.k.n_heads) {
                    r -= a.k.n_heads;
                    part = 2;
                }
            }
            float x[VPL][8];
#pragma unroll
            for (int i = 0; i < VPL; ++i) raw[u][i].get(x[i]);
            if (base + (U + u) * step < nrows) load(u, base + (U + u) * step + sub);
            if (norms) {
                float ss = 0.0f;
#pragma unroll
                for (int i = 0; i < VPL; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) ss = fmaf(x[i][j], x[i][j], ss);
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                if (part == 0 ? a.q_weight != nullptr : part == 1 && a.k_weight) {
                    const float rs = rsqrtf(fmaf(ss, a.inv_dim, a.eps));
#pragma unroll
                    for (int i = 0; i < VPL; ++i)
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            x[i][j] *= rs * (part == 0 ? wq[i][j] : wk[i][j]);
                }
            }
            if (half) {
                if (a.rope.interleaved) {
                    if (part < 2) {
#pragma unroll
                        for (int i = 0; i < VPL; ++i)
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float p = x[i][2 * j], q = x[i][2 * j + 1];
                                x[i][2 * j] = fmaf(p, cs[i][j], -q * sn[i][j]);
                                x[i][2 * j + 1] = fmaf(q, cs[i][j], p * sn[i][j]);
                            }
                    }
                } else {
                    // the other channel of each pair is rot_dim / 2 away: a whole
                    // number of chunks, held by a lane of the same row
                    float y[VPL][8];
#pragma unroll
                    for (int i = 0; i < VPL; ++i) {
                        const int ch = 8 * (col + i * LPR);
                        const int pc = (ch < half ? ch + half : ch - half) / 8;
                        const int from = sub * LPR + ((pc % LPR) + LPR) % LPR;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            if constexpr (VPL == 1) {
                                y[i][j] = __shfl_sync(0xffffffffu, x[0][j], from);
                            } else {
                                y[i][j] = 0.0f;
#pragma unroll
                                for (int v = 0; v < VPL; ++v) {
                                    const float o = __shfl_sync(0xffffffffu, x[v][j], from);
                                    if (pc / LPR == v) y[i][j] = o;
                                }
                            }
                        }
                    }
                    if (part < 2) {
#pragma unroll
                        for (int i = 0; i < VPL; ++i) {
                            if (8 * (col + i * LPR) >= 2 * half) continue;
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                x[i][j] = fmaf(x[i][j], cs[i][j], y[i][j] * sn[i][j]);
                        }
                    }
                }
            }
            if (!PAGED || part == 0) {
                const RowsOut &o = part == 0 ? a.q_out : a.k_out;
                const size_t at = static_cast<size_t>(t * o.stride) +
                                  static_cast<size_t>(r) * a.head_dim;
#pragma unroll
                for (int i = 0; i < VPL; ++i) {
                    const int c = col + i * LPR;
                    if (ok && c < chunks) store8(o.x, o.dtype, at + 8 * c, x[i]);
                }
            }
            if constexpr (PAGED) {
                static_assert(!PAGED || VPL == 1, "paged head dims fit one chunk a lane");
                const size_t row = row0 + static_cast<size_t>(r) * a.cache.page_size;
                void *dst = part == 1 ? a.cache.k : a.cache.v;
                const bool kv = ok && part > 0 && store_kv && col < chunks;
                if (a.cache.dtype == KVD_INT8) {
                    float m = 0.0f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(x[0][j]));
#pragma unroll
                    for (int o = LPR / 2; o > 0; o >>= 1)
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                    const float s = __fdiv_rn(m, 127.0f);
                    uint32_t w[2] = {0, 0};
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        int code = 0;
                        if (s != 0.0f) {
                            code = __float2int_rn(__fdiv_rn(x[0][j], s));
                            code = max(-127, min(127, code));
                        }
                        w[j / 4] |= (static_cast<uint32_t>(code) & 0xffu) << (8 * (j % 4));
                    }
                    if (kv) {
                        *reinterpret_cast<uint2 *>(static_cast<int8_t *>(dst) +
                                                   row * a.head_dim + 8 * col) =
                            make_uint2(w[0], w[1]);
                        if (col == 0)
                            static_cast<float *>(part == 1 ? a.cache.k_scale
                                                           : a.cache.v_scale)[row] = s;
                    }
                } else if (kv) {
                    store8(dst, a.cache.dtype == KVD_BF16 ? KVD_X_BF16 : KVD_X_F16,
                           row * a.head_dim + 8 * col, x[0]);
                }
            }
        }
    }
}

template <typename IN, int LPR, int VPL, int U, bool PAGED>
cudaError_t launch(const RopeArgs &a, cudaStream_t st) {
    const int nrows = a.q.n_heads + a.k.n_heads + a.v.n_heads;
    constexpr int kRows = 32 / LPR;
    // Warps a token: one, or as many as give every SM 16 warps
    const int most = (nrows + kRows - 1) / kRows;
    int parts = (16 * device_sm_count() + a.n_tokens - 1) / a.n_tokens;
    if (parts > most) parts = most;
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
