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
// is cut into pieces of equally many tiles; over its tiles of a head a CTA takes the head's
// rows in tiles of up to 256 (latent rows, whose queries fill more shared memory: 128), the
// queries' tile resident and the keys streaming past it, 64 channels a step.  A key's sum lives
// in `out` between the row tiles, always in the same thread's hands.
//
// Pieces of equally many tiles are pieces of equal work only where every tile is seen by
// equally many row tiles: a batch of single tokens, or of chunks without a window.  A chunk's
// tiles among single tokens', and tiles behind a window, cost their CTA the chunk's row tiles
// or nothing, and the call takes as long as the busiest CTA.  1024 tokens of 32 heads over 8000
// int8 tokens alone 77 us; beside 7 single tokens over 8000 each 467 us, beside 31 over 60,000
// each 9.5 ms (those 32 as single tokens 0.77); 1024 over 60,000 with a window of 4096 454 us.
//
// Measured: single tokens of 32 heads over 8 sequences of 65,536, 8 KV heads, f16 172 us (6.2
// TB/s of keys: HBM), int8 177 us (3.1 TB/s; a tile's way through the turning warps and two
// places, with the issue slots at 38 %); of 64 heads over 16 of 16,384 latent rows 55 us (5.5 TB/s:
// HBM).  1000 tokens of 32 heads over 8000 latent rows 918 us: their 71 tiles occupy 71 CTAs, and
// the keys stream past 250 row tiles of 128 rows.
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

// This CTA's piece of the line; each warp finds it.
__device__ __forceinline__ Line start_of_line(const MassDev &a, bool first_warp, int lane) {
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
    const bool report = blockIdx.x == 0 && first_warp;
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
    return w;
}

// The sum over rows [r0, r1) of 2^(ks * logit + base) of this thread's key; the logits stand
// in `rows` columns of its lane, base is -lse.
__device__ __forceinline__ float weights_of(uint32_t s_at, const float *base, int rows, int r0, int r1,
                                            float ks) {
    float2 acc[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) acc[x] = make_float2(0.0f, 0.0f);
    const float2 k2 = make_float2(ks, ks);
#pragma unroll 1
    for (int c0 = 0; c0 < rows; c0 += 32) {
        float s[32];
        tmem_ld32(s_at + c0, s);
        const bool whole = __all_sync(0xffffffffu, r0 <= c0 && r1 >= c0 + 32);
        tmem_wait_ld();
        pin32(s);
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
            const float4 l = *reinterpret_cast<const float4 *>(base + c0 + c);
            float2 x = __ffma2_rn(make_float2(s[c], s[c + 1]), k2, make_float2(l.x, l.y));
            float2 y = __ffma2_rn(make_float2(s[c + 2], s[c + 3]), k2, make_float2(l.z, l.w));
            s[c] = exp2_approx(x.x);
            s[c + 1] = exp2_approx(x.y);
            s[c + 2] = exp2_approx(y.x);
            s[c + 3] = exp2_approx(y.y);
        }
        if (!whole)
#pragma unroll
            for (int c = 0; c < 32; ++c)
                if (c0 + c < r0 || c0 + c >= r1) s[c] = 0.0f;
#pragma unroll
        for (int c = 0; c < 32; c += 2)
            acc[c / 2 % 4] = __fadd2_rn(acc[c / 2 % 4], make_float2(s[c], s[c + 1]));
    }
#pragma unroll
    for (int x = 1; x < 4; ++x) acc[0] = __fadd2_rn(acc[0], acc[x]);
    return acc[0].x + acc[0].y;
}

// What a weight's exponent begins with, base 2; a row that sees no key has no weights.
__device__ __forceinline__ float base_of(float lse) {
    return lse == -INFINITY ? -INFINITY : -lse * kLog2e;
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
    __shared__ __align__(16) float bases[2][kMaxRows];  // -lse of a row tile, for each team
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

    Line w = start_of_line(a, warp == 0, lane);
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
        const bool again = a.max_new > a.tokens || a.groups > 1;  // keys are read more than once
        const uint64_t policy = again ? l2_policy_evict_last() : l2_policy_evict_first();
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
        float *my_base = bases[team];
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
                        float l = -INFINITY;  // no row there: no weight
                        if (tok < r.cnt && h < r.heads)
                            l = base_of(a.lse[static_cast<int64_t>(g.s.s0 + r.i0 + tok) *
                                                  (a.c.n_kv_heads * a.G) +
                                              g.head * a.G + r.h0 + h]);
                        my_base[x] = l;
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
                        sum += weights_of(s_at, my_base, a.rows, r0, r1, ks);
                        tmem_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bar.s_empty[team]);
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

// ------------------------------------------------------- many rows a KV head ---
// Up to kHeld key tiles stay in shared memory (turned once, where they are int8), and the
// queries stream past them in tiles of 128 rows, so that a product of 128 x 128 costs 8 KB
// of queries where streaming keys would cost 32.  Four warps take a tile of keys each, and
// a thread keeps its key's sum in a register until all rows have passed.
//
// Measured: 1024 tokens of 32 heads over 9024 int8 tokens, 8 KV heads, 79 us: the
// exponentials' pipe at 45 %, the issue slots at 48 %, products 37 %.  With keys streaming past
// resident rows it took 157 us (each tile turned from int8 16 times), and with two teams of
// four warps for the four tiles 126 (two warps a scheduler wait on their own latencies).
constexpr int kHeld = 4;       // and teams of four warps
constexpr int kSumWarps = 4 * kHeld;
constexpr int rows_threads(bool i8) { return 32 * (kSumWarps + (i8 ? 6 : 2)); }
constexpr int kRowsAt = 128;   // rows of a query tile
constexpr int kQueryPlaces = 2;
constexpr int kLseSlots = 8;   // query tiles' statistics

struct RowsBars {
    uint64_t q_full[kQueryPlaces], q_empty[kQueryPlaces], lse_full[kLseSlots], lse_empty[kLseSlots],
        key_full[kHeld], key_raw[kHeld], keys_empty, s_full[kHeld], s_empty[kHeld], done;
};

template <bool BF16, int D, bool I8>
__global__ void __launch_bounds__(rows_threads(I8), 1)
mass_rows_kernel(const __grid_constant__ MassDev a, const __grid_constant__ CUtensorMap q_map,
                 const __grid_constant__ CUtensorMap k_map) {
    constexpr int kChunks = D / 64;
    constexpr int kTileBytes = kChunks * kChunkBytes;      // of 128 rows, keys or queries
    constexpr int kRaw = I8 ? kTileBytes / 2 : 0;          // codes stand in a tile's second half
    extern __shared__ uint8_t raw_smem[];
    __shared__ RowsBars bar;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    __shared__ __align__(16) float bases[kLseSlots][kRowsAt];  // -lse
    uint8_t *keys = raw_smem + ((1024 - (smem_addr(raw_smem) & 1023)) & 1023);
    uint8_t *queries = keys + kHeld * kTileBytes;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (warp == kSumWarps + 1) tmem_alloc(&tmem_slot, 512);
    if (tid == 0) {
        for (int i = 0; i < kQueryPlaces; ++i) {
            mbar_init(&bar.q_full[i], 1);
            mbar_init(&bar.q_empty[i], 1);
        }
        for (int i = 0; i < kLseSlots; ++i) {
            mbar_init(&bar.lse_full[i], 1);
            mbar_init(&bar.lse_empty[i], kSumWarps);
        }
        for (int i = 0; i < kHeld; ++i) {
            mbar_init(&bar.key_full[i], I8 ? 4 : 1);
            mbar_init(&bar.key_raw[i], 1);
        }
        mbar_init(&bar.keys_empty, 1);
        for (int i = 0; i < kHeld; ++i) {
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
    Line w = start_of_line(a, warp == 0, lane);
    const uint32_t tmem = tmem_slot;
    volatile int *abort = &abort_flag;
    auto fail = [&] {
        *abort = 1;
        report_status(a.c.dev_status, KVD_ERR_TIMEOUT);
    };
    Stretch g;
    bool ok = true;

    if (warp == kSumWarps) {
        // ------------------------------------------------------------ loads ---
        const uint64_t policy = l2_policy_evict_first();
        const int boxes = kTile / a.box, ps = a.c.page_size;
        uint32_t chunk = 0, q = 0, asked = 0;  // chunks of key tiles, query tiles, loads of those
        uint32_t loaded[kHeld] = {};         // times each place of keys was loaded
#pragma unroll 1
        while (ok && next_stretch(a, w, g)) {
#pragma unroll 1
            for (int j0 = g.j0; ok && g.row_tiles > 0 && j0 < g.j1; j0 += kHeld, ++chunk) {
                Stretch h = g;
                h.j0 = j0;
                h.j1 = min(j0 + kHeld, g.j1);
                if (chunk > 0 && !(ok = wait_for(&bar.keys_empty, (chunk - 1) & 1, abort))) break;
                // the cache rows of the boxes, a lane a box
                int row = a.dead_row;
                const int t0 = j0 * kTile + lane * a.box;
                if (t0 < h.j1 * kTile && t0 < g.s.len) {
                    const int col = t0 / ps, page = checked_page(a.c, g.b, col);
                    if (page >= 0)
                        row = (page * a.c.n_kv_heads + g.head) * ps + (t0 - col * ps);
                }
                const int mine = lane / boxes;  // tile of the chunk, 4 x 8 boxes at most
#pragma unroll
                for (int t = 0; t < kHeld; ++t) {
                    if (j0 + t >= h.j1) break;
                    uint64_t *full = I8 ? &bar.key_raw[t] : &bar.key_full[t];
                    if (lane == 0) mbar_arrive_expect_tx(full, I8 ? kTile * D : kTileBytes);
                    ++loaded[t];
                    __syncwarp();
                    if (mine == t) {
                        uint8_t *dst = keys + t * kTileBytes;
                        const int at = lane % boxes * a.box;
                        if constexpr (I8) {
                            tma_load_2d(dst + kRaw + at * D, &k_map, 0, row, full, policy);
                        } else {
#pragma unroll
                            for (int c = 0; c < kChunks; ++c)
                                tma_load_2d(dst + c * kChunkBytes + at * 128, &k_map, c * 64, row,
                                            full, policy);
                        }
                    }
                    __syncwarp();
                }
#pragma unroll 1
                for (int i = 0; i < g.row_tiles; ++i) {
                    const RowTile r = row_tile(a, h, i);
                    if (r.ja == r.jb) continue;
                    // the rows' statistics, on their way
                    float l[kRowsAt / 32];
#pragma unroll
                    for (int x = 0; x < kRowsAt / 32; ++x) {
                        const int at = x * 32 + lane, tok = at / a.heads;
                        l[x] = -INFINITY;  // no row there: no weight
                        if (tok < r.cnt)
                            l[x] = a.lse[static_cast<int64_t>(g.s.s0 + r.i0 + tok) *
                                             (a.c.n_kv_heads * a.G) +
                                         g.head * a.G + at - tok * a.heads];
                    }
                    const uint32_t st = q % kQueryPlaces, round = q / kQueryPlaces;
                    if (round > 0 && !(ok = wait_for(&bar.q_empty[st], (round - 1) & 1, abort))) break;
                    ++asked;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&bar.q_full[st], kChunks * a.heads * a.tokens * 128);
#pragma unroll
                        for (int c = 0; c < kChunks; ++c)
                            tma_load_4d(queries + st * kTileBytes + c * kChunkBytes, &q_map, c * 64, 0,
                                        g.head, g.s.s0 + r.i0, &bar.q_full[st]);
                    }
                    if (q >= kLseSlots &&
                        !(ok = wait_for(&bar.lse_empty[q % kLseSlots], (q / kLseSlots - 1) & 1, abort)))
                        break;
#pragma unroll
                    for (int x = 0; x < kRowsAt / 32; ++x)
                        bases[q % kLseSlots][x * 32 + lane] = base_of(l[x]);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.lse_full[q % kLseSlots]);
                    ++q;
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
#pragma unroll
            for (int t = 0; t < kHeld; ++t)
                if (landed && loaded[t] > 0)
                    landed = mbar_wait(I8 ? &bar.key_raw[t] : &bar.key_full[t], (loaded[t] - 1) & 1, &none);
            for (uint32_t i = 0; landed && i < kQueryPlaces; ++i) {
                const uint32_t fills = (asked + kQueryPlaces - 1 - i) / kQueryPlaces;
                if (fills > 0) landed = mbar_wait(&bar.q_full[i], (fills - 1) & 1, &none);
            }
        }
        return;
    } else if (warp == kSumWarps + 1) {
        // -------------------------------------------------- products S^T = K Q^T ---
        constexpr uint32_t kIdS = mma_idesc(BF16, kTile, kRowsAt, false);
        const uint32_t k_base = warp_uniform(desc_low(smem_addr(keys), 16));
        const uint32_t q_base = warp_uniform(desc_low(smem_addr(queries), 16));
        const uint32_t tmem_u = warp_uniform(tmem);
        uint32_t q = 0, loaded[kHeld] = {}, used = 0;  // used: bits, of the tiles' logits
#pragma unroll 1
        while (ok && next_stretch(a, w, g)) {
#pragma unroll 1
            for (int j0 = g.j0; ok && g.row_tiles > 0 && j0 < g.j1; j0 += kHeld) {
                Stretch h = g;
                h.j0 = j0;
                h.j1 = min(j0 + kHeld, g.j1);
#pragma unroll
                for (int t = 0; t < kHeld; ++t)
                    if (ok && j0 + t < h.j1) ok = wait_for(&bar.key_full[t], loaded[t]++ & 1, abort);
                if (!ok) break;
#pragma unroll 1
                for (int i = 0; ok && i < g.row_tiles; ++i) {
                    const RowTile r = row_tile(a, h, i);
                    if (r.ja == r.jb) continue;
                    const uint32_t st = q % kQueryPlaces;
                    if (!(ok = wait_for(&bar.q_full[st], (q / kQueryPlaces) & 1, abort))) break;
                    ++q;
                    const uint32_t qd = warp_uniform(q_base + st * (kTileBytes / 16));
#pragma unroll 1
                    for (int j = r.ja; j < r.jb; ++j) {
                        const int t = j - j0;
                        // (the first wait of a barrier's life ends at once)
                        if (!(ok = wait_for(&bar.s_empty[t], ~(used >> t) & 1, abort))) break;
                        used ^= 1u << t;
                        tmem_fence_after();
                        const uint32_t s_at = warp_uniform(tmem_u + t * kRowsAt);
                        const uint32_t k = warp_uniform(k_base + t * (kTileBytes / 16));
                        if (elect_one()) {
#pragma unroll
                            for (int x = 0; x < D / 16; ++x) {
                                const uint32_t at = (x / 4 * kChunkBytes + x % 4 * 32) / 16;
                                mma_ss(s_at, smem_desc(k + at), smem_desc(qd + at), kIdS, x > 0);
                            }
                            mma_commit(&bar.s_full[t]);
                            if (j + 1 == r.jb) mma_commit(&bar.q_empty[st]);
                        }
                        __syncwarp();
                    }
                }
                if (elect_one()) mma_commit(&bar.keys_empty);
                __syncwarp();
            }
        }
        if (!ok) fail();
        // every product and every barrier arrival is done before the CTA goes
        if (elect_one()) mma_commit(&bar.done);
        __syncwarp();
        volatile int none = 0;
        if (!mbar_wait(&bar.done, 0, &none)) fail();
    } else if (I8 && warp > kSumWarps + 1) {
        // ------------------------------------------------ int8 to f16 or bf16 ---
        // In place: all four warps hold a tile's codes in registers before they write.
        constexpr int kUnits = D / 16;
        constexpr int kRows = 32 / kUnits * 4;  // rows of a step of the four warps
        constexpr int kSteps = kTile / kRows;
        const int q8 = lane >> 3, k8 = lane & 7;
        const int row = (warp - kSumWarps - 2) * (32 / kUnits) +
                        (D == 128 ? 2 * (q8 >> 1) + (k8 >> 2) : lane >> 2);
        const int u = D == 128 ? (k8 & 3) + 4 * ((q8 & 1) ^ (k8 >> 2)) : lane & 3;
        const int dst_row = (u / 4) * kChunkBytes + row * 128;
        const int dst0 = dst_row + 16 * (((u % 4) * 2) ^ (row & 7));
        const int dst1 = dst_row + 16 * (((u % 4) * 2 + 1) ^ (row & 7));
        static_assert(kRows % 8 == 0, "the swizzle of a lane's row stays");
        uint32_t loaded[kHeld] = {};
#pragma unroll 1
        while (next_stretch(a, w, g)) {
#pragma unroll 1
            for (int j0 = g.j0; g.row_tiles > 0 && j0 < g.j1; j0 += kHeld) {
#pragma unroll
                for (int t = 0; t < kHeld; ++t) {
                    if (j0 + t >= g.j1) break;
                    // (none of the four leaves before the others: they meet below)
                    if (ok) ok = wait_for(&bar.key_raw[t], loaded[t] & 1, abort);
                    ++loaded[t];
                    uint8_t *tile = keys + t * kTileBytes;
                    const uint8_t *src = tile + kRaw + row * D + 16 * u;
                    uint4 v[kSteps];
#pragma unroll
                    for (int x = 0; x < kSteps; ++x)
                        v[x] = *reinterpret_cast<const uint4 *>(src + x * (kRows * D));
                    asm volatile("bar.sync 3, 128;" ::: "memory");
#pragma unroll
                    for (int x = 0; x < kSteps; ++x) {
                        uint4 lo, hi;
                        codes_to<BF16>(v[x].x, lo.x, lo.y);
                        codes_to<BF16>(v[x].y, lo.z, lo.w);
                        codes_to<BF16>(v[x].z, hi.x, hi.y);
                        codes_to<BF16>(v[x].w, hi.z, hi.w);
                        *reinterpret_cast<uint4 *>(tile + dst0 + x * (kRows * 128)) = lo;
                        *reinterpret_cast<uint4 *>(tile + dst1 + x * (kRows * 128)) = hi;
                    }
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.key_full[t]);
                }
            }
        }
        if (!ok) fail();
    } else if (warp < kSumWarps) {
        // --------------------------------------------------------------- sums ---
        const int team = warp >> 2, key = tid & 127;
        const uint32_t s_at = tmem + ((warp & 3) << 21) + team * kRowsAt;
        uint32_t n = 0, q = 0;  // this team's products, query tiles
#pragma unroll 1
        while (ok && next_stretch(a, w, g)) {
            const size_t row = static_cast<size_t>(g.b) * a.c.n_kv_heads + g.head;
            const int ps = a.c.page_size;
#pragma unroll 1
            for (int j0 = g.j0; ok && j0 < g.j1; j0 += kHeld) {
                Stretch h = g;
                h.j0 = j0;
                h.j1 = min(j0 + kHeld, g.j1);
                // this thread's key: what stands there, its scale, whether it counts
                const int j = j0 + team, t = j * kTile + key;
                const bool here = j < h.j1 && t < g.s.len;
                float sum = 0.0f, ks = a.scale_log2;
                bool some = false;
                if (here) {
                    const int page = a.c.page_table[static_cast<size_t>(g.b) * a.c.max_pages + t / ps];
                    some = page >= 0 && page < a.c.n_pages;
                    if (I8 && some)
                        ks *= static_cast<const float *>(
                            a.c.k_scale)[(static_cast<size_t>(page) * a.c.n_kv_heads + g.head) * ps +
                                         t % ps];
                    if (a.mass && t < g.s.first) sum = a.decay * a.mass[row * a.mass_stride + t];
                }
#pragma unroll 1
                for (int i = 0; i < g.row_tiles; ++i) {
                    const RowTile r = row_tile(a, h, i);
                    if (r.ja == r.jb) continue;
                    const uint32_t slot = q % kLseSlots;
                    if (!(ok = wait_for(&bar.lse_full[slot], (q / kLseSlots) & 1, abort))) break;
                    ++q;
                    if (j >= r.ja && j < r.jb) {
                        // the rows [r0, r1) that see this key
                        int r0 = 0, r1 = 0;
                        if (some && t >= r.lo && t < r.hi) {
                            const int f = max(t - r.p0, 0);
                            int l = r.cnt - 1;
                            if (a.window > 0) l = min(l, t + a.window - 1 - r.p0);
                            if (f <= l) {
                                r0 = f * a.heads;
                                r1 = (l + 1) * a.heads;
                            }
                        }
                        if (!(ok = wait_for(&bar.s_full[team], n & 1, abort))) break;
                        ++n;
                        tmem_fence_after();
                        sum += weights_of(s_at, bases[slot], kRowsAt, r0, r1, ks);
                        tmem_fence_before();
                    }
                    __syncwarp();
                    if (lane == 0) {
                        if (j >= r.ja && j < r.jb) mbar_arrive(&bar.s_empty[team]);
                        mbar_arrive(&bar.lse_empty[slot]);
                    }
                }
                if (here) a.sums[row * a.sums_stride + t] = sum;
            }
        }
        if (!ok) fail();
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == kSumWarps + 1) {
        tmem_fence_after();
        tmem_free(tmem, 512);
    }
}

struct Maps {
    CUtensorMap q, k;
};

// The arguments that both kernels take; row tiles of whole tokens of a group of heads, up to
// `most` rows.
bool fill(const MassArgs &m, int most, MassDev &a, Maps &maps) {
    const PagedAttnArgs &p = m.attn;
    const kvd_paged_cache &c = p.c;
    const bool i8 = c.dtype == KVD_INT8;
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
    const int G = p.G > 0 ? p.G : 1;
    a.groups = (G + most - 1) / most;
    a.heads = (G + a.groups - 1) / a.groups;
    a.tokens = most / a.heads;
    if (a.tokens > p.max_new && p.max_new > 0) a.tokens = p.max_new;
    a.rows = (a.heads * a.tokens + 15) / 16 * 16;

    const cuuint64_t W = static_cast<cuuint64_t>(c.head_dim);
    const cuuint64_t kd[2] = {W, static_cast<cuuint64_t>(pool)};
    const cuuint64_t ks[1] = {W * (i8 ? 1 : 2)};
    const cuuint32_t kb[2] = {i8 ? static_cast<cuuint32_t>(W) : 64, static_cast<cuuint32_t>(a.box)};
    if (!make_map(&maps.k, c.dtype, c.k, 2, kd, ks, kb,
                  i8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B))
        return false;
    if (!p.starts) return true;
    const cuuint64_t qd[4] = {W, static_cast<cuuint64_t>(G), static_cast<cuuint64_t>(c.n_kv_heads),
                              static_cast<cuuint64_t>(p.n_tokens)};
    const cuuint64_t qs[3] = {W * 2, W * 2 * G, static_cast<cuuint64_t>(p.q_stride) * 2};
    const cuuint32_t qb[4] = {64, static_cast<cuuint32_t>(a.heads), 1,
                              static_cast<cuuint32_t>(a.tokens)};
    return make_map(&maps.q, p.bf16 ? KVD_BF16 : KVD_F16, p.q, 4, qd, qs, qb);
}

template <bool BF16, int I8>
cudaError_t launch_type(const MassArgs &m, cudaStream_t st) {
    MassDev a = {};
    Maps maps = {};
    if (!fill(m, m.attn.c.head_dim <= 128 ? kMaxRows : 128, a, maps)) return cudaErrorInvalidValue;
    a.per = a.chunks <= 2 ? a.chunks : 1;
    a.raws = I8 ? 4 : 0;
    const int q_bytes = a.chunks * a.rows * 128, place = a.per * kChunkBytes;
    const int rest = 222 * 1024 - q_bytes - a.raws * kTile * I8;
    a.places = rest / place < kMaxPlaces ? rest / place : kMaxPlaces;
    if (I8 && a.places > 2) a.places = 2;
    const size_t smem = 1024 + q_bytes + static_cast<size_t>(a.places) * place + a.raws * kTile * I8;
    auto *kernel = mass_kernel<BF16, I8>;
    constexpr int threads = I8 ? 448 : 320;
    cudaError_t e = prepare_kernel(reinterpret_cast<const void *>(kernel), threads, smem);
    if (e != cudaSuccess) return e;
    return launch_ex(kernel, dim3(device_sm_count()), dim3(threads), smem, st, true, a, maps.q, maps.k);
}

template <bool BF16, int D, bool I8>
cudaError_t launch_many(const MassArgs &m, cudaStream_t st) {
    MassDev a = {};
    Maps maps = {};
    if (!fill(m, kRowsAt, a, maps)) return cudaErrorInvalidValue;
    constexpr size_t smem = 1024 + (kHeld + kQueryPlaces) * static_cast<size_t>(D / 64 * kChunkBytes);
    auto *kernel = mass_rows_kernel<BF16, D, I8>;
    constexpr int threads = rows_threads(I8);
    cudaError_t e = prepare_kernel(reinterpret_cast<const void *>(kernel), threads, smem);
    if (e != cudaSuccess) return e;
    return launch_ex(kernel, dim3(device_sm_count()), dim3(threads), smem, st, true, a, maps.q, maps.k);
}

template <bool BF16>
cudaError_t launch_q(const MassArgs &m, cudaStream_t st) {
    const kvd_paged_cache &c = m.attn.c;
    // More rows than a tile that stays: the keys stay instead.  With the attention, over 60,000
    // f16 tokens, 8 KV heads: 260 rows a head 169 us against 193 with keys that stream, 512 rows
    // 183 and 178, 2048 604 and 641; the limit at 64 rows instead: 132 rows 122 us against 102.
    // The rule is the batch's, by its longest run of new tokens: a chunk sends the single tokens
    // beside it to the kernel whose keys stay, too.
    const bool many = c.head_dim <= 128 && static_cast<int64_t>(m.attn.G) * m.attn.max_new > kMaxRows;
    if (c.dtype == KVD_INT8) {
        if (c.head_dim == 64)
            return many ? launch_many<BF16, 64, true>(m, st) : launch_type<BF16, 64>(m, st);
        return many ? launch_many<BF16, 128, true>(m, st) : launch_type<BF16, 128>(m, st);
    }
    if (!many) return launch_type<BF16, 0>(m, st);
    return c.head_dim == 64 ? launch_many<BF16, 64, false>(m, st)
                            : launch_many<BF16, 128, false>(m, st);
}

}  // namespace

cudaError_t launch_mass(const MassArgs &a, cudaStream_t st) {
    // (without queries the type of the keys' products is any)
    const bool bf16 = a.attn.c.dtype == KVD_BF16 || a.attn.bf16;
    return bf16 ? launch_q<true>(a, st) : launch_q<false>(a, st);
}

}  // namespace kvd
