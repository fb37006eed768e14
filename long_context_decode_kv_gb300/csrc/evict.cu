// evict.cu -- dropping tokens of a paged cache by the weight that attention gave them
// (kvd_paged_evict, kvd_latent_evict): which ones stay, then their rows to other pages.
//
// choose_kernel, a cluster a (sequence, head): the n-th largest weight by its bits, 11, 11
// and 10 at a time (a histogram of each block's slice in shared memory, summed over the
// cluster through it), then the kept tokens in order, each warp counting its run of
// tokens before it writes them.  The weights are read once, into shared memory, where a
// slice fits it.
//
// move_kernel: a warp looks up 16 rows' places, a lane a row, and copies them 16 bytes a
// lane with all its loads in flight.  The rows go to other pages than they come from
// (which other sequences may share), so no order between the copies matters.
#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"
#include "paged.h"
#include "paged_dev.cuh"

namespace kvd {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kCached = 16384;  // weights a block keeps in shared memory
constexpr int kBins = 2048;

// Larger weight, larger key; NaN below all.
__device__ __forceinline__ uint32_t weight_key(float w) {
    return w != w ? 0u : float_to_key(w);
}

__global__ void __launch_bounds__(kThreads)
choose_kernel(const __grid_constant__ EvictArgs a, int blocks) {
    extern __shared__ uint32_t cached[];
    __shared__ uint32_t hist[2][kBins];
    __shared__ int warp_sum[kWarps], warp_gt[kWarps], warp_eq[kWarps];
    __shared__ int found_bin, found_above;
    __shared__ int total_gt, total_eq;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(blockIdx.x) % blocks;
    const int row = static_cast<int>(blockIdx.x) / blocks;  // of a sequence and a head
    const int b = row / a.c.n_kv_heads;
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
    // those that stay whatever they weigh
    for (int t = rank * kThreads + tid; t < lo; t += blocks * kThreads) put(t, t, mass[t]);
    for (int t = hi + rank * kThreads + tid; t < L; t += blocks * kThreads)
        put(n - (L - t), t, mass[t]);
    int need = n - lo - (L - hi);
    if (need <= 0) return;  // the same for the whole cluster

    // this block's slice of the others
    const int slice = ((hi - lo + blocks - 1) / blocks + kThreads - 1) / kThreads * kThreads;
    const int t0 = min(lo + rank * slice, hi), count = min(slice, hi - t0);
    const bool fits = slice <= kCached;
    for (int i = tid; i < 2 * kBins; i += kThreads) (&hist[0][0])[i] = 0;
    if (fits)
        for (int i = tid; i < count; i += kThreads) cached[i] = weight_key(mass[t0 + i]);
    __syncthreads();
    auto key_of = [&](int i) { return fits ? cached[i] : weight_key(mass[t0 + i]); };

    uint32_t prefix = 0, mask = 0;  // the bits of the n-th largest found so far
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : kBins;
        uint32_t *h = hist[pass & 1];
#pragma unroll 4
        for (int i = tid; i < count; i += kThreads) {
            const uint32_t k = key_of(i);
            if ((k & mask) == prefix) atomicAdd(&h[(k >> shift) & (bins - 1)], 1u);
        }
        cluster.sync();
        // the buffer of the pass before is free: its readers have come to this barrier
        if (pass == 1)
            for (int i = tid; i < kBins; i += kThreads) hist[0][i] = 0;
        // bins from the top, 4 a thread: where the sum passes `need`
        constexpr int kEach = kBins / kThreads;
        int at[kEach], sum = 0;
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const int bin = bins - 1 - (tid * kEach + j);
            at[j] = 0;
            if (bin >= 0)
                for (int r = 0; r < blocks; ++r)
                    at[j] += static_cast<int>(*cluster.map_shared_rank(&h[bin], r));
            sum += at[j];
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
        for (int w = 0; w < warp; ++w) above += warp_sum[w];
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            if (above < need && above + at[j] >= need) {
                found_bin = bins - 1 - (tid * kEach + j);
                found_above = above;
            }
            above += at[j];
        }
        __syncthreads();
        need -= found_above;
        prefix |= static_cast<uint32_t>(found_bin) << shift;
        mask |= static_cast<uint32_t>(bins - 1) << shift;
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
    if (tid == 0) {
        int g = 0, e = 0;
        for (int w = 0; w < kWarps; ++w) {
            g += warp_gt[w];
            e += warp_eq[w];
        }
        total_gt = g;
        total_eq = e;
    }
    cluster.sync();
    gt = eq = 0;
    for (int r = 0; r < rank; ++r) {
        gt += *cluster.map_shared_rank(&total_gt, r);
        eq += *cluster.map_shared_rank(&total_eq, r);
    }
    cluster.sync();  // no block goes while others read from it
    for (int w = 0; w < warp; ++w) {
        gt += warp_gt[w];
        eq += warp_eq[w];
    }
    const uint32_t below = (1u << lane) - 1;
#pragma unroll 1
    for (int i = i0; i < i1; i += 32) {
        const bool in = i + lane < i1;
        const uint32_t k = in ? key_of(i + lane) : 0u;
        const bool is_gt = in && k > prefix, is_eq = in && k == prefix;
        const uint32_t gts = __ballot_sync(0xffffffffu, is_gt);
        const uint32_t eqs = __ballot_sync(0xffffffffu, is_eq);
        const int my_eq = eq + __popc(eqs & below);
        if (is_gt || (is_eq && my_eq < need)) {
            const int t = t0 + i + lane;
            put(a.sink + gt + __popc(gts & below) + min(my_eq, need), t, mass[t]);
        }
        gt += __popc(gts);
        eq += __popc(eqs);
    }
}

constexpr int kMoveRows = 16;  // a warp's
constexpr int kMoveThreads = 128;

__global__ void __launch_bounds__(kMoveThreads)
move_kernel(const __grid_constant__ EvictArgs a, int64_t units, int per_row) {
    const int lane = threadIdx.x & 31;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * (kMoveThreads / 32);
    const int vecs = a.row_bytes / 16;
    const int ps = a.c.page_size, Hkv = a.c.n_kv_heads;
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kMoveThreads / 32) + (threadIdx.x >> 5);
         u < units; u += stride) {
        const int row = static_cast<int>(u / per_row);
        const int r0 = static_cast<int>(u % per_row) * kMoveRows;
        const int b = row / Hkv, g = row - b * Hkv;
        const int n = min(a.keep, min(max(a.c.seq_lens[b], 0), a.c.len));
        if (r0 >= n) continue;
        const int rows = min(kMoveRows, n - r0);
        int64_t src = -1, dst = -1;  // cache rows
        if (lane < rows) {
            const int t = a.kept[static_cast<size_t>(row) * a.keep + r0 + lane], r = r0 + lane;
            const int from = checked_page(a.c, b, t / ps);
            const int to = a.to[static_cast<size_t>(b) * a.to_cols + r / ps];
            if (to < 0 || to >= a.c.n_pages) {
                report_status(a.c.dev_status, KVD_ERR_INVALID);
            } else if (from >= 0) {
                src = (static_cast<int64_t>(from) * Hkv + g) * ps + t % ps;
                dst = (static_cast<int64_t>(to) * Hkv + g) * ps + r % ps;
                if (a.c.k_scale) {
                    float *ks = static_cast<float *>(a.c.k_scale);
                    float *vs = static_cast<float *>(a.c.v_scale);
                    ks[dst] = ks[src];
                    vs[dst] = vs[src];
                }
            }
        }
        const int total = rows * vecs, step_r = 32 / vecs, step_v = 32 % vecs;
        auto copy = [&](uint8_t *base) {
            int r = lane / vecs, v = lane % vecs;
            constexpr int U = 8;
            for (int i0 = 0; i0 < total; i0 += 32 * U) {
                uint4 x[U];
                int64_t to[U];
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    const int64_t s = __shfl_sync(0xffffffffu, src, r & 31);
                    const int64_t d = __shfl_sync(0xffffffffu, dst, r & 31);
                    to[j] = r < rows && d >= 0 ? d * a.row_bytes + 16 * v : -1;
                    if (to[j] >= 0)
                        x[j] = __ldcs(reinterpret_cast<const uint4 *>(base + s * a.row_bytes + 16 * v));
                    r += step_r;
                    v += step_v;
                    if (v >= vecs) {
                        v -= vecs;
                        ++r;
                    }
                }
#pragma unroll
                for (int j = 0; j < U; ++j)
                    if (to[j] >= 0) *reinterpret_cast<uint4 *>(base + to[j]) = x[j];
            }
        };
        copy(static_cast<uint8_t *>(a.c.k));
        if (a.c.v) copy(static_cast<uint8_t *>(a.c.v));
    }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs &a, cudaStream_t st) {
    // blocks a (sequence, head): up to 8, each with 2048 tokens at least
    int blocks = 1;
    while (blocks < kMaxCluster && a.c.len > blocks * 2048) blocks *= 2;
    const int rows = a.c.batch * a.c.n_kv_heads;
    const size_t smem = kCached * sizeof(uint32_t);
    cudaError_t e = prepare_kernel(reinterpret_cast<const void *>(choose_kernel), kThreads, smem);
    if (e != cudaSuccess) return e;
    e = launch_cluster(choose_kernel, dim3(rows * blocks), dim3(kThreads), blocks, smem, st, a, blocks);
    if (e != cudaSuccess) return e;
    const int most = a.keep < a.c.len ? a.keep : a.c.len;
    const int per_row = (most + kMoveRows - 1) / kMoveRows;
    const int64_t units = static_cast<int64_t>(rows) * per_row;
    const int64_t want = (units + kMoveThreads / 32 - 1) / (kMoveThreads / 32);
    const int64_t grid = want < 64ll * device_sm_count() ? want : 64ll * device_sm_count();
    if (grid == 0) return cudaSuccess;
    return launch_ex(move_kernel, dim3(static_cast<unsigned>(grid)), dim3(kMoveThreads), 0, st, true,
                     a, units, per_row);
}

}  // namespace kvd
