// mass.cu -- accumulated attention weight of each cached token (kvd_paged_mass,
// kvd_latent_mass):
//
//   out_t = (old ? decay mass_t : 0) + sum over rows r that see t of exp(scale q_r . k_t - lse_r)
//
// The rows' statistics lse come from the attention call, so the keys are read once and
// no maximum is looked for.  Keys take the tensor core's 128 lanes and the rows its
// columns, S^T = K Q^T: a thread holds one key, and adds its rows' weights up in its own
// registers, so that no sum crosses threads, and none is joined between CTAs.
//
// One CTA per SM, persistent.  The line of all (sequence, KV head) key tiles of 128 tokens
// is cut into equal pieces; over its tiles of a head a CTA takes the head's rows in tiles
// of up to 256 (latent rows, whose queries fill more shared memory: 128), the queries'
// tile resident and the keys streaming past it, 64 channels a step.  A key's sum lives in
// `out` between the row tiles, always in the same thread's hands.
//
// Roles: warps 0-3 and 4-7 take the tiles of even and odd index, a thread a key; warp 8
// loads by TMA, warp 9 issues the products; int8: warps 10-13 turn codes into f16 or bf16
// whole numbers, and the key's scale multiplies its logits.
#include "paged_attn_dev.cuh"

namespace kvd {
namespace {

constexpr int kChunkBytes = kTile * 128;  // 64 channels of a key tile
constexpr int kMaxRows = 256;             // of a row tile
constexpr int kMaxPlaces = 12;

struct MassDev : AttnArgs {
    const float *mass;
    float *sums;
    int64_t mass_stride, sums_stride;
    float decay;
    int chunks, per;        // 64-channel chunks of a key, and of them in a place of the ring
    int places, raws;       // places of the ring, and (int8) of the ring of codes
    int rows;               // of a row tile, a multiple of 16
    int heads, groups, tokens;  // a row tile: heads of a KV head (of so many groups), tokens
};

struct Line {  // a CTA's walk along the line of key tiles
    int b, head, off, left;
    Seq s;
};
struct Stretch {  // tiles [j0, j1) of a (sequence, head)
    int b, head, j0, j1;
    Seq s;
    int row_tiles;
};
struct RowTile {
    int i0, cnt, h0, heads;  // tokens of the sequence's new ones, heads
    int p0;                  // position of the first
    int lo, hi;              // keys that some of its rows see
    int ja, jb;              // the stretch's tiles with such keys
};

__device__ __forceinline__ Seq mass_seq(const MassDev &a, int b, bool report) {
    if (a.starts) return seq_of(a, b, report);
    const int len = min(max(a.c.seq_lens[b], 0), a.c.len);
    if (report && len != a.c.seq_lens[b]) report_status(a.c.dev_status, KVD_ERR_INVALID);
    return Seq{0, 0, len, len};
}
__device__ __forceinline__ int tiles_of(const Seq &s) { return (s.len + kTile - 1) / kTile; }

__device__ __forceinline__ bool next_stretch(const MassDev &a, Line &w, Stretch &g) {
    if (w.left <= 0) return false;
    const int take = min(tiles_of(w.s) - w.off, w.left);
    g.b = w.b;
    g.head = w.head;
    g.j0 = w.off;
    g.j1 = w.off + take;
    g.s = w.s;
    g.row_tiles = (w.s.n + a.tokens - 1) / a.tokens * a.groups;
    w.left -= take;
    w.off = 0;
    if (w.left > 0 && ++w.head == a.c.n_kv_heads) {
        w.head = 0;
#pragma unroll 1
        do {
            if (++w.b >= a.c.batch) {
                w.left = 0;
                break;
            }
            w.s = mass_seq(a, w.b, false);
        } while (w.s.len == 0);
    }
    return true;
}

__device__ __forceinline__ RowTile row_tile(const MassDev &a, const Stretch &g, int i) {
    RowTile r;
    const int tok = i / a.groups;
    r.i0 = tok * a.tokens;
    r.cnt = min(a.tokens, g.s.n - r.i0);
    r.h0 = (i - tok * a.groups) * a.heads;
    r.heads = min(a.heads, a.G - r.h0);
    r.p0 = g.s.first + r.i0;
    r.hi = max(r.p0 + r.cnt, 0);
    r.lo = a.window > 0 ? min(max(r.p0 - a.window + 1, 0), r.hi) : 0;
    r.ja = max(g.j0, r.lo / kTile);
    r.jb = max(min(g.j1, (r.hi + kTile - 1) / kTile), r.ja);
    return r;
}

struct MassBars {
    uint64_t q_full, q_empty, full[kMaxPlaces], empty[kMaxPlaces], raw_full[4], raw_empty[4],
        s_full[2], s_empty[2], done;
};

// I8: 0, or the channels of a row of codes (64 or 128)
template <bool BF16, int I8>
__global__ void __launch_bounds__(I8 ? 448 : 320, 1)
mass_kernel(const __grid_constant__ MassDev a, const __grid_constant__ CUtensorMap q_map,
            const __grid_constant__ CUtensorMap k_map) {
    extern __shared__ uint8_t raw_smem[];
    __shared__ MassBars bar;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    __shared__ __align__(16) float lse[2][kMaxRows];  // of a row tile, base 2, for each team
    uint8_t *smem = raw_smem + ((1024 - (smem_addr(raw_smem) & 1023)) & 1023);
    uint8_t *q_smem = smem;
    uint8_t *ring = smem + a.chunks * a.rows * 128;
    const int place_bytes = a.per * kChunkBytes;
    uint8_t *raws = ring + a.places * place_bytes;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (warp == 9) tmem_alloc(&tmem_slot, 512);
    if (tid == 0) {
        mbar_init(&bar.q_full, 1);
        mbar_init(&bar.q_empty, 1);
        for (int i = 0; i < kMaxPlaces; ++i) {
            mbar_init(&bar.full[i], I8 ? 4 : 1);
            mbar_init(&bar.empty[i], 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&bar.raw_full[i], 1);
            mbar_init(&bar.raw_empty[i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.s_full[i], 1);
            mbar_init(&bar.s_empty[i], 4);
        }
        mbar_init(&bar.done, 1);
        fence_barrier_init();
        abort_flag = 0;
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    pdl_wait();
    pdl_launch_dependents();

    // ---- this CTA's piece of the line, found by each warp
    auto cost_of = [&](int b, bool report) -> int {
        return b < a.c.batch ? tiles_of(mass_seq(a, b, report)) * a.c.n_kv_heads : 0;
    };
    auto scan = [&](int v) -> int {  // inclusive
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        return v;
    };
    const bool report = blockIdx.x == 0 && warp == 0;
    int cost = cost_of(lane, report);
    int upto = scan(cost);
    int total = __shfl_sync(0xffffffffu, upto, 31);
#pragma unroll 1
    for (int b0 = 32; b0 < a.c.batch; b0 += 32)
        total += __reduce_add_sync(0xffffffffu, cost_of(b0 + lane, report));
    const int ctas = min(static_cast<int>(gridDim.x), total);
    Line w;
    w.left = 0;
    if (static_cast<int>(blockIdx.x) < ctas) {
        const int share = total / ctas, spare = total % ctas, c = blockIdx.x;
        const int x0 = c * share + min(c, spare);
        int base = 0;
#pragma unroll 1
        for (int b0 = 0;; b0 += 32) {
            if (b0 > 0) {
                cost = cost_of(b0 + lane, false);
                upto = scan(cost);
            }
            const uint32_t in =
                __ballot_sync(0xffffffffu, cost > 0 && base + upto - cost <= x0 && x0 < base + upto);
            if (in) {
                const int l = __ffs(in) - 1;
                w.b = b0 + l;
                const int r = x0 - base - __shfl_sync(0xffffffffu, upto - cost, l);
                w.s = mass_seq(a, w.b, false);
                const int tiles = tiles_of(w.s);
                w.head = r / tiles;
                w.off = r - w.head * tiles;
                w.left = share + (c < spare ? 1 : 0);
                break;
            }
            base += __shfl_sync(0xffffffffu, upto, 31);
            if (b0 + 32 >= a.c.batch) break;
        }
    }
    const uint32_t tmem = tmem_slot;
    volatile int *abort = &abort_flag;
    auto fail = [&] {
        *abort = 1;
        report_status(a.c.dev_status, KVD_ERR_TIMEOUT);
    };
    Stretch g;
    bool ok = true;
    const int places = a.places, steps = a.chunks / a.per;  // places a key tile takes

    if (warp == 8) {
        // ------------------------------------------------------------ loads ---
        const uint64_t policy = a.max_new > a.tokens ? l2_policy_evict_last() : l2_policy_evict_first();
        const int boxes = kTile / a.box, ps = a.c.page_size;
        const int per_read = 32 / boxes;  // tiles whose rows one read of the page table gives
        uint32_t st = 0, round = 0, queries = 0;
        const int ring_places = I8 ? a.raws : places;
        uint64_t *full = I8 ? bar.raw_full : bar.full, *empty = I8 ? bar.raw_empty : bar.empty;
#pragma unroll 1
        while (ok && next_stretch(a, w, g)) {
#pragma unroll 1
            for (int i = 0; ok && i < g.row_tiles; ++i) {
                const RowTile r = row_tile(a, g, i);
                if (r.ja == r.jb) continue;
                if (queries > 0 && !(ok = wait_for(&bar.q_empty, (queries - 1) & 1, abort))) break;
                ++queries;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&bar.q_full, a.chunks * a.heads * a.tokens * 128);
#pragma unroll 1
                    for (int c = 0; c < a.chunks; ++c)
                        tma_load_4d(q_smem + c * a.rows * 128, &q_map, c * 64, r.h0, g.head,
                                    g.s.s0 + r.i0, &bar.q_full);
                }
                __syncwarp();
                // the cache rows of the boxes of tiles j, j + 1, .., a lane a box
                auto rows_of = [&](int j) -> int {
                    const int t0 = (j + lane / boxes) * kTile + lane % boxes * a.box;
                    if (t0 >= r.jb * kTile || t0 >= g.s.len) return a.dead_row;
                    const int col = t0 / ps;
                    const int page = checked_page(a.c, g.b, col);
                    return page < 0 ? a.dead_row
                                    : (page * a.c.n_kv_heads + g.head) * ps + (t0 - col * ps);
                };
                int rows = 0, rows_next = rows_of(r.ja);
#pragma unroll 1
                for (int j = r.ja; ok && j < r.jb; ++j) {
                    const int in = (j - r.ja) % per_read;
                    if (in == 0) {
                        rows = rows_next;
                        rows_next = rows_of(j + per_read);
                    }
                    const int row = __shfl_sync(0xffffffffu, rows, in * boxes + lane % boxes);
#pragma unroll 1
                    for (int step = 0; step < (I8 ? 1 : steps); ++step) {
                        if (round > 0 && !(ok = wait_for(&empty[st], (round - 1) & 1, abort))) break;
                        if (lane == 0)
                            mbar_arrive_expect_tx(&full[st], I8 ? kTile * I8 : place_bytes);
                        __syncwarp();
                        if (lane < boxes) {
                            if constexpr (I8 > 0) {
                                tma_load_2d(raws + st * (kTile * I8) + lane * a.box * I8, &k_map, 0,
                                            row, &full[st], policy);
                            } else {
#pragma unroll 1
                                for (int c = 0; c < a.per; ++c)
                                    tma_load_2d(ring + st * place_bytes + c * kChunkBytes +
                                                    lane * a.box * 128,
                                                &k_map, (step * a.per + c) * 64, row, &full[st],
                                                policy);
                            }
                        }
                        if (++st == static_cast<uint32_t>(ring_places)) {
                            st = 0;
                            ++round;
                        }
                    }
                }
            }
        }
        if (!ok) fail();
        tmem_fence_before();
        __syncthreads();  // all roles are done, and know whether a wait ran out
        if (*abort) {
            // nothing may land in shared memory after the CTA has gone
            volatile int none = 0;
            bool landed = true;  // after one wait that runs out all has had the time to land
            for (int i = 0; landed && i < ring_places; ++i) {
                const uint32_t fills = round + (static_cast<uint32_t>(i) < st ? 1 : 0);
                if (fills > 0) landed = mbar_wait(&full[i], (fills - 1) & 1, &none);
            }
            if (landed && queries > 0) mbar_wait(&bar.q_full, (queries - 1) & 1, &none);
        }
        return;
    } else if (warp == 9) {
        // -------------------------------------------------- products S^T = K Q^T ---
        const uint32_t idesc = warp_uniform(mma_idesc(BF16, kTile, 16, false) +
                                            (static_cast<uint32_t>(a.rows / 8 - 2) << 17));
        const uint32_t ring_addr = smem_addr(ring);
        const uint32_t q = warp_uniform(desc_low(smem_addr(q_smem), 16));
        const uint32_t q_chunk = warp_uniform(a.rows * 128 / 16);
        const uint32_t tmem_u = warp_uniform(tmem);
        uint32_t st = 0, round = 0, queries = 0, used[2] = {0, 0};
#pragma unroll 1
        while (ok && next_stretch(a, w, g)) {
#pragma unroll 1
            for (int i = 0; ok && i < g.row_tiles; ++i) {
                const RowTile r = row_tile(a, g, i);
                if (r.ja == r.jb) continue;
                if (!(ok = wait_for(&bar.q_full, queries & 1, abort))) break;
                ++queries;
#pragma unroll 1
                for (int j = r.ja; ok && j < r.jb; ++j) {
                    const int team = j & 1;
                    const uint32_t n = team ? used[1]++ : used[0]++;
                    if (n > 0 && !(ok = wait_for(&bar.s_empty[team], (n - 1) & 1, abort))) break;
                    tmem_fence_after();
                    const uint32_t s_at = warp_uniform(tmem_u + team * kMaxRows);
#pragma unroll 1
                    for (int step = 0; step < steps; ++step) {
                        if (!(ok = wait_for(&bar.full[st], round & 1, abort))) break;
                        tmem_fence_after();
                        const uint32_t k = warp_uniform(desc_low(ring_addr + st * place_bytes, 16));
                        if (elect_one()) {
#pragma unroll 1
                            for (int c = 0; c < a.per; ++c)
#pragma unroll
                                for (int x = 0; x < 4; ++x)
                                    mma_ss(s_at, smem_desc(k + (c * kChunkBytes + x * 32) / 16),
                                           smem_desc(q + (step * a.per + c) * q_chunk + x * 2), idesc,
                                           step > 0 || c > 0 || x > 0);
                            mma_commit(&bar.empty[st]);
                            if (step + 1 == steps) mma_commit(&bar.s_full[team]);
                            if (step + 1 == steps && j + 1 == r.jb) mma_commit(&bar.q_empty);
                        }
                        __syncwarp();
                        if (++st == static_cast<uint32_t>(places)) {
                            st = 0;
                            ++round;
                        }
                    }
                }
            }
        }
        if (!ok) fail();
        // every product and every barrier arrival is done before the CTA goes
        if (elect_one()) mma_commit(&bar.done);
        __syncwarp();
        volatile int none = 0;
        if (!mbar_wait(&bar.done, 0, &none)) fail();
    } else if (I8 && warp >= 10) {
        // ------------------------------------------------ int8 to f16 or bf16 ---
        // A lane's row and 16 codes of a step: the 8 lanes of a load or a store lie on
        // two rows, at 128 channels on the one's first half and the other's second, so
        // that the codes come from all banks; and as the swizzle turns even chunks of an
        // odd row into odd ones, the chunks go to all banks too.
        constexpr int D = I8 ? I8 : 64;
        constexpr int kUnits = D / 16;
        constexpr int kRows = 32 / kUnits * 4;  // rows of a step of the four warps
        constexpr int kSteps = kTile / kRows;
        const int q8 = lane >> 3, k8 = lane & 7;
        const int row = (warp - 10) * (32 / kUnits) +
                        (D == 128 ? 2 * (q8 >> 1) + (k8 >> 2) : lane >> 2);
        const int u = D == 128 ? (k8 & 3) + 4 * ((q8 & 1) ^ (k8 >> 2)) : lane & 3;
        const int dst_row = (u / 4) * kChunkBytes + row * 128;
        const int dst0 = dst_row + 16 * (((u % 4) * 2) ^ (row & 7));
        const int dst1 = dst_row + 16 * (((u % 4) * 2 + 1) ^ (row & 7));
        static_assert(kRows % 8 == 0, "the swizzle of a lane's row stays");
        uint32_t rs = 0, raw_round = 0, st = 0, round = 0;
#pragma unroll 1
        while (ok && next_stretch(a, w, g)) {
#pragma unroll 1
            for (int i = 0; ok && i < g.row_tiles; ++i) {
                const RowTile r = row_tile(a, g, i);
#pragma unroll 1
                for (int j = r.ja; j < r.jb; ++j) {
                    if (!(ok = wait_for(&bar.raw_full[rs], raw_round & 1, abort))) break;
                    if (round > 0 && !(ok = wait_for(&bar.empty[st], (round - 1) & 1, abort))) break;
                    const uint8_t *src = raws + rs * (kTile * D) + row * D + 16 * u;
                    uint8_t *dst = ring + st * place_bytes;
#pragma unroll 4
                    for (int x = 0; x < kSteps; ++x) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(src + x * (kRows * D));
                        uint4 lo, hi;
                        codes_to<BF16>(v.x, lo.x, lo.y);
                        codes_to<BF16>(v.y, lo.z, lo.w);
                        codes_to<BF16>(v.z, hi.x, hi.y);
                        codes_to<BF16>(v.w, hi.z, hi.w);
                        *reinterpret_cast<uint4 *>(dst + dst0 + x * (kRows * 128)) = lo;
                        *reinterpret_cast<uint4 *>(dst + dst1 + x * (kRows * 128)) = hi;
                    }
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&bar.full[st]);
                        mbar_arrive(&bar.raw_empty[rs]);
                    }
                    if (++rs == static_cast<uint32_t>(a.raws)) {
                        rs = 0;
                        ++raw_round;
                    }
                    if (++st == static_cast<uint32_t>(places)) {
                        st = 0;
                        ++round;
                    }
                }
            }
        }
        if (!ok) fail();
    } else if (warp < 8) {
        // --------------------------------------------------------------- sums ---
        const int team = warp >> 2, key = tid & 127;
        const uint32_t s_at = tmem + ((warp & 3) << 21) + team * kMaxRows;
        float *my_lse = lse[team];
        uint32_t n = 0;
        // A team's warps meet at barriers of the hardware, which have no limit: so none
        // leaves its loops before the others, and a wait that ran out only makes the waits
        // behind it pass.
        auto meet = [&] { asm volatile("bar.sync %0, 128;" ::"r"(1 + team) : "memory"); };
#pragma unroll 1
        while (next_stretch(a, w, g)) {
            const size_t row = static_cast<size_t>(g.b) * a.c.n_kv_heads + g.head;
            float *sums = a.sums + row * a.sums_stride;
            const float *mass = a.mass ? a.mass + row * a.mass_stride : nullptr;
            const int32_t *table = a.c.page_table + static_cast<size_t>(g.b) * a.c.max_pages;
            const int ps = a.c.page_size;
            const int first_j = g.j0 + ((g.j0 ^ team) & 1);
            auto page_of = [&](int j) -> int {
                const int t = j * kTile + key;
                return t < g.s.len && j < g.j1 ? table[t / ps] : -1;
            };
#pragma unroll 1
            for (int i = 0; i < max(g.row_tiles, 1); ++i) {
                RowTile r = {};
                if (i < g.row_tiles) r = row_tile(a, g, i);
                if (r.ja < r.jb) {
                    meet();  // the rows before have been read
                    for (int x = key; x < a.rows; x += 128) {
                        const int tok = x / a.heads, h = x - tok * a.heads;
                        float l = INFINITY;  // no row there: no weight
                        if (tok < r.cnt && h < r.heads) {
                            l = a.lse[static_cast<int64_t>(g.s.s0 + r.i0 + tok) *
                                          (a.c.n_kv_heads * a.G) +
                                      g.head * a.G + r.h0 + h] *
                                kLog2e;
                            if (l == -INFINITY) l = INFINITY;
                        }
                        my_lse[x] = l;
                    }
                    meet();
                }
                // the first row tile's pass sets what no row sees too
                int j = i == 0 ? first_j : r.ja + ((r.ja ^ team) & 1);
                const int end = i == 0 ? g.j1 : r.jb;
                int page_next = page_of(j);
#pragma unroll 1
                for (; j < end; j += 2) {
                    const int t = j * kTile + key, page = page_next;
                    page_next = page_of(j + 2);
                    const bool bad = page < 0 || page >= a.c.n_pages;  // or no token
                    float sum = 0.0f, ks = a.scale_log2;
                    if (I8 && !bad)
                        ks *= static_cast<const float *>(
                            a.c.k_scale)[(static_cast<size_t>(page) * a.c.n_kv_heads + g.head) * ps +
                                         t % ps];
                    if (t < g.s.len) {
                        if (i > 0)
                            sum = sums[t];
                        else if (mass && t < g.s.first)
                            sum = a.decay * mass[t];
                    }
                    if (j >= r.ja && j < r.jb) {
                        // the rows [r0, r1) that see this key
                        int r0 = 0, r1 = 0;
                        if (!bad && t >= r.lo && t < r.hi) {
                            const int f = max(t - r.p0, 0);
                            int l = r.cnt - 1;
                            if (a.window > 0) l = min(l, t + a.window - 1 - r.p0);
                            if (f <= l) {
                                r0 = f * a.heads;
                                r1 = (l + 1) * a.heads;
                            }
                        }
                        if (ok) ok = wait_for(&bar.s_full[team], n & 1, abort);
                        ++n;
                        tmem_fence_after();
                        float2 acc[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x) acc[x] = make_float2(0.0f, 0.0f);
                        const float2 k2 = make_float2(ks, ks);
                        auto add = [&](const float *s, int c0) {
                            const bool whole =
                                __all_sync(0xffffffffu, r0 <= c0 && r1 >= c0 + 32);
#pragma unroll
                            for (int c = 0; c < 32; c += 4) {
                                const float4 l = *reinterpret_cast<const float4 *>(my_lse + c0 + c);
                                float2 x = __ffma2_rn(make_float2(s[c], s[c + 1]), k2,
                                                      make_float2(-l.x, -l.y));
                                float2 y = __ffma2_rn(make_float2(s[c + 2], s[c + 3]), k2,
                                                      make_float2(-l.z, -l.w));
                                x = make_float2(exp2_approx(x.x), exp2_approx(x.y));
                                y = make_float2(exp2_approx(y.x), exp2_approx(y.y));
                                if (!whole) {
                                    const int at = c0 + c;
                                    if (at < r0 || at >= r1) x.x = 0.0f;
                                    if (at + 1 < r0 || at + 1 >= r1) x.y = 0.0f;
                                    if (at + 2 < r0 || at + 2 >= r1) y.x = 0.0f;
                                    if (at + 3 < r0 || at + 3 >= r1) y.y = 0.0f;
                                }
                                acc[c / 4 % 2] = __fadd2_rn(acc[c / 4 % 2], x);
                                acc[2 + c / 4 % 2] = __fadd2_rn(acc[2 + c / 4 % 2], y);
                            }
                        };
                        float s0[32], s1[32];
                        tmem_ld32(s_at, s0);
#pragma unroll 1
                        for (int c = 0; c < a.rows; c += 64) {
                            tmem_wait_ld();
                            pin32(s0);
                            if (c + 32 < a.rows) tmem_ld32(s_at + c + 32, s1);
                            add(s0, c);
                            tmem_wait_ld();
                            pin32(s1);
                            if (c + 64 < a.rows) tmem_ld32(s_at + c + 64, s0);
                            if (c + 32 < a.rows) add(s1, c + 32);
                        }
                        tmem_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bar.s_empty[team]);
#pragma unroll
                        for (int x = 1; x < 4; ++x) acc[0] = __fadd2_rn(acc[0], acc[x]);
                        sum += acc[0].x + acc[0].y;
                    }
                    if (t < g.s.len) sums[t] = sum;
                }
            }
        }
        if (!ok) fail();
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == 9) {
        tmem_fence_after();
        tmem_free(tmem, 512);
    }
}

template <bool BF16, int I8>
cudaError_t launch_type(const MassArgs &m, cudaStream_t st) {
    const PagedAttnArgs &p = m.attn;
    const kvd_paged_cache &c = p.c;
    MassDev a = {};
    a.c = c;
    a.G = p.G;
    a.n_tokens = p.n_tokens;
    a.max_new = p.max_new;
    a.window = p.window;
    a.starts = p.starts;
    a.scale_log2 = p.scale_log2;
    a.lse = p.lse;
    a.mass = m.mass;
    a.sums = m.out;
    a.mass_stride = m.mass_stride;
    a.sums_stride = m.out_stride;
    a.decay = m.decay;
    a.box = 16;
    while (a.box < kTile && c.page_size % (2 * a.box) == 0) a.box *= 2;
    const int64_t pool = static_cast<int64_t>(c.n_pages) * c.n_kv_heads * c.page_size;
    a.dead_row = static_cast<int>(pool);
    a.chunks = (c.head_dim + 63) / 64;
    // Row tiles: whole tokens of a group of heads
    const int most = a.chunks <= 2 ? kMaxRows : 128;
    const int G = p.G > 0 ? p.G : 1;
    a.groups = (G + most - 1) / most;
    a.heads = (G + a.groups - 1) / a.groups;
    a.tokens = most / a.heads;
    if (a.tokens > p.max_new && p.max_new > 0) a.tokens = p.max_new;
    a.rows = (a.heads * a.tokens + 15) / 16 * 16;
    a.per = a.chunks <= 2 ? a.chunks : 1;
    a.raws = I8 ? 4 : 0;
    const int q_bytes = a.chunks * a.rows * 128, place = a.per * kChunkBytes;
    const int rest = 222 * 1024 - q_bytes - a.raws * kTile * I8;
    a.places = rest / place < kMaxPlaces ? rest / place : kMaxPlaces;
    if (I8 && a.places > 2) a.places = 2;
    const size_t smem = 1024 + q_bytes + static_cast<size_t>(a.places) * place + a.raws * kTile * I8;

    CUtensorMap q_map = {}, k_map;
    const cuuint64_t W = static_cast<cuuint64_t>(c.head_dim);
    const cuuint64_t kd[2] = {W, static_cast<cuuint64_t>(pool)};
    const cuuint64_t ks[1] = {W * (I8 ? 1 : 2)};
    const cuuint32_t kb[2] = {I8 ? static_cast<cuuint32_t>(I8) : 64, static_cast<cuuint32_t>(a.box)};
    if (!make_map(&k_map, c.dtype, c.k, 2, kd, ks, kb,
                  I8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    if (p.starts) {
        const cuuint64_t qd[4] = {W, static_cast<cuuint64_t>(G), static_cast<cuuint64_t>(c.n_kv_heads),
                                  static_cast<cuuint64_t>(p.n_tokens)};
        const cuuint64_t qs[3] = {W * 2, W * 2 * G, static_cast<cuuint64_t>(p.q_stride) * 2};
        const cuuint32_t qb[4] = {64, static_cast<cuuint32_t>(a.heads), 1,
                                  static_cast<cuuint32_t>(a.tokens)};
        if (!make_map(&q_map, BF16 ? KVD_BF16 : KVD_F16, p.q, 4, qd, qs, qb))
            return cudaErrorInvalidValue;
    }
    auto *kernel = mass_kernel<BF16, I8>;
    constexpr int threads = I8 ? 448 : 320;
    cudaError_t e = prepare_kernel(reinterpret_cast<const void *>(kernel), threads, smem);
    if (e != cudaSuccess) return e;
    return launch_ex(kernel, dim3(device_sm_count()), dim3(threads), smem, st, true, a, q_map, k_map);
}

}  // namespace

cudaError_t launch_mass(const MassArgs &a, cudaStream_t st) {
    const kvd_paged_cache &c = a.attn.c;
    if (c.dtype == KVD_INT8) {
        if (c.head_dim == 64)
            return a.attn.bf16 ? launch_type<true, 64>(a, st) : launch_type<false, 64>(a, st);
        return a.attn.bf16 ? launch_type<true, 128>(a, st) : launch_type<false, 128>(a, st);
    }
    return c.dtype == KVD_BF16 ? launch_type<true, 0>(a, st) : launch_type<false, 0>(a, st);
}

}  // namespace kvd
