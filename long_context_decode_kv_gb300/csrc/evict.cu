// evict.cu -- dropping tokens of a paged cache by the weight that attention gave them
// (kvd_paged_evict, kvd_latent_evict): which ones stay, then their rows to other pages.
//
// choose_kernel, a cluster a (sequence, head): the n-th largest weight by its bits, 11, 11
// and 10 at a time until a bin's keys stay as one (a histogram of each block's slice in
// shared memory, added up in the first block's), then the kept tokens in order, each warp
// counting its run of tokens before it writes them.  The weights are read once, into shared
// memory, where a slice fits it.
//
// Measured, 8 sequences of up to 65,536 int8 tokens and 8 heads cut to 16,384: 107 us, of
// which moving takes 72 (6.4 TB/s, 0.95 of what a copy reaches) and choosing the rest, in
// passes of 4 us with a meeting of the cluster each (with the keys read four at a time it
// took 6 more).  4096 tokens of 8 heads to 1024: 13.6 us.  One sequence of 1,048,576 of 8 int8
// heads to 4096: 300 us, nearly all of it the choice (8 blocks a row, 64 in all, which read their
// slices in every pass).
//
// move_kernel: a warp looks up 32 rows' places, a lane a row, and copies them 16 bytes a
// lane, 8 loads in flight.  The rows go to other pages than they come from
// (which other sequences may share), so no order between the copies matters.  Latent rows
// (72 parts of 16 bytes at 576 channels, a lane's row and part counted on the way): 8 sequences
// of 65,536 to 16,384 98 us with the choice, the moves at 4.3 TB/s.
#include <cooperative_groups.h>

#include <utility>

#include "common.cuh"
#include "internal.h"
#include "paged.h"
#include "paged_dev.cuh"

namespace kvd {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
// Weights a block keeps in shared memory: as many as leave room for two blocks an SM (64 KB
// beside 33 KB of histograms; a row's 4 or 8 blocks wait for one another between short passes, and
// a second block fills the waits).  Longer slices are read again in each pass.  With the moves, 64
// rows cut to a quarter: of 131,072 weights 295 us (8192 weights a block 349, 32,768 376, 49,152
// 421), of 262,144 584 (688, 754, 845); of 65,536 and 8 rows of 1,048,576 the larger ones are no
// faster, and 8192 takes 182 us for 130 and 617 for 566.
constexpr int kCached = 16384;
constexpr int kBins = 2048;

// Larger weight, larger key; NaN below all.
__device__ __forceinline__ uint32_t weight_key(float w) {
    return w != w ? 0u : float_to_key(w);
}

__global__ void __launch_bounds__(kThreads)
choose_kernel(const __grid_constant__ EvictArgs a, int blocks, int room) {
    extern __shared__ uint32_t cached[];  // `room` keys
    __shared__ uint32_t hist[kBins];
    __shared__ __align__(16) uint32_t total[3][kBins];  // of the cluster, in its first block
    __shared__ int warp_sum[kWarps], warp_gt[kWarps], warp_eq[kWarps];
    __shared__ int found_bin, found_above, found_count;
    __shared__ int block_gt[kMaxCluster], block_eq[kMaxCluster];  // in each block
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(blockIdx.x) % blocks;
    const int row = static_cast<int>(blockIdx.x) / blocks;  // of a sequence and a head
    const int b = row / a.c.n_kv_heads;
    for (int i = tid; i < kBins; i += kThreads) hist[i] = total[0][i] = total[1][i] = total[2][i] = 0;
    auto cleared = cluster.barrier_arrive();
    pdl_wait();
    pdl_launch_dependents();
    const int L = checked_len(a.c, b);
    const int n = min(a.keep, L);
    const float *mass = a.mass + static_cast<size_t>(row) * a.mass_stride;
    int32_t *kept = a.kept + static_cast<size_t>(row) * a.keep;
    float *mass_out = a.mass_out ? a.mass_out + static_cast<size_t>(row) * a.mass_out_stride : nullptr;
    if (rank == 0 && tid == 0 && row % a.c.n_kv_heads == 0) a.lens_out[b] = n;
    auto put = [&](int at, int t, float w) {
        kept[at] = t;
        if (mass_out) mass_out[at] = w;
    };
    const int lo = L <= a.keep ? L : a.sink, hi = L <= a.keep ? L : L - a.recent;
    // this block's slice of those between, on its way
    int need = n - lo - (L - hi);
    const int slice = ((hi - lo + blocks - 1) / blocks + kThreads - 1) / kThreads * kThreads;
    const int t0 = min(lo + rank * slice, hi), count = min(slice, hi - t0);
    const bool fits = slice <= room;
    if (need > 0 && fits)
#pragma unroll 16
        for (int i = tid; i < count; i += kThreads) cached[i] = weight_key(mass[t0 + i]);
    // those that stay whatever they weigh
    for (int t = rank * kThreads + tid; t < lo; t += blocks * kThreads) put(t, t, mass[t]);
    for (int t = hi + rank * kThreads + tid; t < L; t += blocks * kThreads)
        put(n - (L - t), t, mass[t]);
    cluster.barrier_wait(std::move(cleared));  // the sums are clear, in the first block too
    if (need <= 0) return;                     // the same for the whole cluster
    auto key_of = [&](int i) { return fits ? cached[i] : weight_key(mass[t0 + i]); };
    if (fits) __syncthreads();

    uint32_t prefix = 0, mask = 0;  // the bits of the n-th largest found so far
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : kBins;
#pragma unroll 8
        for (int i = tid; i < count; i += kThreads) {
            const uint32_t k = key_of(i);
            if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & (bins - 1)], 1u);
        }
        __syncthreads();
        uint32_t *sums = cluster.map_shared_rank(&total[pass][0], 0);
#pragma unroll
        for (int i = tid; i < kBins; i += kThreads) {
            const uint32_t v = hist[i];
            if (v) {
                atomicAdd(&sums[i], v);
                hist[i] = 0;
            }
        }
        cluster.sync();
        // bins from the top, 4 a thread: where the sum passes `need`
        constexpr int kEach = kBins / kThreads;
        static_assert(kEach == 4, "read as one vector");
        const int bottom = bins - kEach * (tid + 1);
        int at[kEach] = {}, sum = 0;
        if (bottom >= 0) {
            const uint4 v = *reinterpret_cast<const uint4 *>(&sums[bottom]);
            at[0] = v.w;
            at[1] = v.z;
            at[2] = v.y;
            at[3] = v.x;
            sum = at[0] + at[1] + at[2] + at[3];
        }
        int upto = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += u;
        }
        if (lane == 31) warp_sum[warp] = upto;
        __syncthreads();
        int above = upto - sum;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            if (w < warp) above += warp_sum[w];
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            if (above < need && above + at[j] >= need) {
                found_bin = bins - 1 - (tid * kEach + j);
                found_above = above;
                found_count = at[j];
            }
            above += at[j];
        }
        __syncthreads();
        need -= found_above;
        prefix |= static_cast<uint32_t>(found_bin) << shift;
        mask |= static_cast<uint32_t>(bins - 1) << shift;
        if (found_count == need && prefix > 0) {
            // all with these bits stay: those above the largest key below them
            --prefix;
            need = 0;
            break;
        }
    }
    // Kept: keys above prefix, and the first `need` of those equal to it.
    const int run = slice / kWarps, i0 = warp * run, i1 = min(i0 + run, count);
    int gt = 0, eq = 0;
#pragma unroll 4
    for (int i = i0 + lane; i < i1; i += 32) {
        const uint32_t k = key_of(i);
        gt += k > prefix;
        eq += k == prefix;
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) {
        warp_gt[warp] = gt;
        warp_eq[warp] = eq;
    }
    __syncthreads();
    if (tid < blocks) {  // the block's counts to every block
        int g = 0, e = 0;
        for (int w = 0; w < kWarps; ++w) {
            g += warp_gt[w];
            e += warp_eq[w];
        }
        *cluster.map_shared_rank(&block_gt[rank], tid) = g;
        *cluster.map_shared_rank(&block_eq[rank], tid) = e;
    }
    cluster.sync();  // (after it no block's memory is another's business)
    gt = eq = 0;
    for (int r = 0; r < rank; ++r) {
        gt += block_gt[r];
        eq += block_eq[r];
    }
    for (int w = 0; w < warp; ++w) {
        gt += warp_gt[w];
        eq += warp_eq[w];
    }
    const uint32_t below = (1u << lane) - 1;
#pragma unroll 2
    for (int i = i0; i < i1; i += 32) {
        const bool in = i + lane < i1;
        const uint32_t k = in ? key_of(i + lane) : 0u;
        const bool is_gt = in && k > prefix, is_eq = in && k == prefix;
        const uint32_t gts = __ballot_sync(0xffffffffu, is_gt);
        const uint32_t eqs = __ballot_sync(0xffffffffu, is_eq);
        const int my_eq = eq + __popc(eqs & below);
        if (is_gt || (is_eq && my_eq < need)) {
            const int t = t0 + i + lane;
            // (0: it was NaN)
            put(a.sink + gt + __popc(gts & below) + min(my_eq, need), t,
                k == 0 ? mass[t] : key_to_float(k));
        }
        gt += __popc(gts);
        eq += __popc(eqs);
    }
}

constexpr int kMoveRows = 32;  // a warp's
constexpr int kMoveThreads = 128;

// VECS: 16-byte parts of a row of k, and of v (0: any number, of k alone)
template <int VECS>
__global__ void __launch_bounds__(kMoveThreads)
move_kernel(const __grid_constant__ EvictArgs a, int64_t units, int per_row) {
    const int lane = threadIdx.x & 31;
    const int ps = a.c.page_size, Hkv = a.c.n_kv_heads;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * (kMoveThreads / 32);
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kMoveThreads / 32) + (threadIdx.x >> 5);
         u < units; u += stride) {
        const int row = static_cast<int>(u / per_row);
        const int r0 = static_cast<int>(u % per_row) * kMoveRows;
        const int b = row / Hkv, g = row - b * Hkv;
        const int n = min(a.keep, min(max(a.c.seq_lens[b], 0), a.c.len));
        if (r0 >= n) continue;
        int src = -1, dst = -1;  // cache rows (the pool has fewer than 2^31)
        if (r0 + lane < n) {
            const int r = r0 + lane;
            const int t = __ldcs(a.kept + static_cast<size_t>(row) * a.keep + r);
            const int to = a.to[static_cast<size_t>(b) * a.to_cols + r / ps];
            const int from = checked_page(a.c, b, t / ps);
            if (to < 0 || to >= a.c.n_pages) {
                report_status(a.c.dev_status, KVD_ERR_INVALID);
            } else if (from >= 0) {
                src = (from * Hkv + g) * ps + t % ps;
                dst = (to * Hkv + g) * ps + r % ps;
            }
        }
        float k_scale = 0.0f, v_scale = 0.0f;
        if (a.c.k_scale && dst >= 0) {
            k_scale = static_cast<float *>(a.c.k_scale)[src];
            v_scale = static_cast<float *>(a.c.v_scale)[src];
        }
        uint4 *k = static_cast<uint4 *>(a.c.k), *v = static_cast<uint4 *>(a.c.v);
        if constexpr (VECS > 0) {
            // a step: 32 / VECS rows of k and v; U steps' reads are under way together
            constexpr int kAt = 32 / VECS, U = VECS < 4 ? VECS : 4;
            const int part = lane % VECS;
#pragma unroll 1
            for (int i = 0; i < VECS; i += U) {
                uint4 x[U], y[U];
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    const int s = __shfl_sync(0xffffffffu, src, (i + j) * kAt + lane / VECS);
                    if (s >= 0) {
                        x[j] = __ldcs(k + static_cast<size_t>(s) * VECS + part);
                        y[j] = __ldcs(v + static_cast<size_t>(s) * VECS + part);
                    }
                }
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    const int d = __shfl_sync(0xffffffffu, dst, (i + j) * kAt + lane / VECS);
                    if (d >= 0) {
                        k[static_cast<size_t>(d) * VECS + part] = x[j];
                        v[static_cast<size_t>(d) * VECS + part] = y[j];
                    }
                }
            }
        } else {
            const int vecs = a.row_bytes / 16, rows = min(kMoveRows, n - r0);
            constexpr int U = 8;
            const int total = rows * vecs, step_r = 32 / vecs, step_v = 32 % vecs;
            int r = lane / vecs, part = lane % vecs;
#pragma unroll 1
            for (int i = 0; i < total; i += 32 * U) {
                uint4 x[U];
                const int was_r = r, was_part = part;
                auto next = [&] {
                    r += step_r;
                    part += step_v;
                    if (part >= vecs) {
                        part -= vecs;
                        ++r;
                    }
                };
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    const int s = __shfl_sync(0xffffffffu, src, r & 31);
                    if (r < rows && s >= 0) x[j] = __ldcs(k + static_cast<size_t>(s) * vecs + part);
                    next();
                }
                r = was_r;
                part = was_part;
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    const int d = __shfl_sync(0xffffffffu, dst, r & 31);
                    if (r < rows && d >= 0) k[static_cast<size_t>(d) * vecs + part] = x[j];
                    next();
                }
            }
        }
        if (a.c.k_scale && dst >= 0) {
            static_cast<float *>(a.c.k_scale)[dst] = k_scale;
            static_cast<float *>(a.c.v_scale)[dst] = v_scale;
        }
    }
}

template <int VECS>
cudaError_t launch_move(const EvictArgs &a, int rows, cudaStream_t st) {
    const int most = a.keep < a.c.len ? a.keep : a.c.len;
    const int per_row = (most + kMoveRows - 1) / kMoveRows;
    const int64_t units = static_cast<int64_t>(rows) * per_row;
    const int64_t want = (units + kMoveThreads / 32 - 1) / (kMoveThreads / 32);
    const int64_t grid = want < (1 << 20) ? want : 1 << 20;
    if (grid == 0) return cudaSuccess;
    return launch_ex(move_kernel<VECS>, dim3(static_cast<unsigned>(grid)), dim3(kMoveThreads), 0, st,
                     true, a, units, per_row);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs &a, cudaStream_t st) {
    // Blocks a (sequence, head): as many as give each 1024 tokens and are all resident at
    // once.  64 rows of 65,536 tokens: 4 blocks 109 us with the moves, 8 (two waves) 128; 8 rows
    // of 4096: 4 blocks 14.9 us, 1, 2 and 8 blocks 17.7, 15.3 to 16.3 and 17.0.
    const int rows = a.c.batch * a.c.n_kv_heads;
    int blocks = kMaxCluster, room = 0, occ = 1;
    size_t smem = 0;
    cudaError_t e;
    for (;; blocks /= 2) {
        const int slice = ((a.c.len + blocks - 1) / blocks + kThreads - 1) / kThreads * kThreads;
        room = slice < kCached ? slice : kCached;
        smem = room * sizeof(uint32_t);
        e = prepare_kernel(reinterpret_cast<const void *>(choose_kernel), kThreads, smem, &occ);
        if (e != cudaSuccess) return e;
        if (blocks == 1 || (a.c.len > 1024 * (blocks / 2) &&
                            static_cast<int64_t>(rows) * blocks <= static_cast<int64_t>(occ) * device_sm_count()))
            break;
    }
    e = launch_cluster(choose_kernel, dim3(rows * blocks), dim3(kThreads), blocks, smem, st, a, blocks,
                       room);
    if (e != cudaSuccess) return e;
    const int vecs = a.c.v ? a.row_bytes / 16 : 0;
    if (vecs == 4) return launch_move<4>(a, rows, st);
    if (vecs == 8) return launch_move<8>(a, rows, st);
    if (vecs == 16) return launch_move<16>(a, rows, st);
    return launch_move<0>(a, rows, st);
}

}  // namespace kvd
