// latent_attn.cu -- attention of a ragged batch's new tokens over a paged cache of latent
// rows, which all query heads share (kvd_latent_attn):
//
//   z_t = scale q . row_t (R + P channels),  out = sum_t softmax(z)_t row_t[:R],
//   p - window < t <= p
//
// A row is key and value at once, so it comes into shared memory once and both products
// read it there.  An output row has R = 512 channels in f32: 128 of them would fill the
// tensor memory and leave none for the logits.  So the rows (tokens' query heads) stand
// on the products' narrow side, up to 64 of them,
//   S^T = K Q^T   64 keys x rows          O^T += V^T P^T   128 channels x rows, R / 128 times
// with S of four tiles and O in 4 * 64 + 4 * 64 columns, and key tiles are 64 tokens, of which
// two fit beside the queries (72 KB each at 576 channels).  Measured, clocks a product
// of 16: 64 x 64 32, 128 x 64 48 (shared memory's rate; 128 x 128 64): 1920 for 64 rows
// and 64 keys of 576 channels, 1.35 PFLOP/s at most.
//
// One CTA per SM, persistent.  An item is a run of a sequence's new tokens, with its heads
// up to 64 rows, over the key tiles that any of them sees.  All items' key tiles form one
// line, cut into equal costs for the CTAs; an item that a cut divides is joined from f32
// partials by join_kernel.  More than 64 heads are so many groups, and the CTAs teams of one
// a group, which walk the same piece of the line at the same time: a key tile comes from
// HBM once, and from the L2 for the others.
//
// Roles: warps 0-3 and 4-7 softmax of the rows' first and second half, a thread 2 keys and
// an eighth of the rows (the layout of 16 x 256-bit reads from tensor memory, of which
// 64-lane products fill 16 lanes a warp); warp 8 issues S^T, warp 9 O^T, warps 10 and 11
// load by TMA (a copy's issue takes a warp some 100 clocks, and pages of 16 tokens take 36 of
// them a tile; with one, two and three warps 24 ragged sequences took 111, 96 and 96 us, 4 x
// 100,000 tokens 87, 86 and 90).  Asking the L2 for the tiles that follow made the calls
// that HBM bounds slower: 94 us 2 tiles ahead, 101 us 6 ahead.  A key tile's places are released
// 128 channels at a time, as O^T is done with them.
//
// The reference m of a row's weights 2^(logit - m) follows its maximum loosely, from kLift
// places below it, as in paged_decode.cu: no search for a tile's maximum unless a weight
// passes kRedo.  P is rounded to the cache's type (half a step of each weight); sums and
// statistics are f32.
//
// Measured, rows of 512 + 64 channels.  1000 tokens of 32 heads over 8000: 695 us, 0.85
// PFLOP/s; shared memory bounds it (operands 63 % of its cycles, tiles coming in 20 %, the
// softmax 7 %), with the tensor pipe at 54 %.  32 tokens of 128 heads over 8192 each: 110 us,
// the same bound and the starts and ends of segments.  4 tokens of 32 heads over 100,000: 85
// us, 5.4 TB/s, HBM and the latency of two tiles a CTA.  One token of 16 heads over 512: 14.6
// us, two launches.  Slower: two key tiles a softmax step (465 us for 424 at 256 + 64
// channels, 1000 tokens over 8000), and two softmax teams that take turns with the references
// (718 us for 694 at 512 + 64, 489 for 417 at 256 + 64).
#include <cstddef>

#include "paged_attn_dev.cuh"

namespace kvd {
namespace {

constexpr int kKeys = 64;              // keys a tile
constexpr int kHalf = kKeys * 128;     // 64 channels of it
constexpr int kPair = 2 * kHalf;       // 128 channels
constexpr int kMaxRing = 8;            // tiles in shared memory
constexpr int kMaxTops = 4;            // 128-channel parts of the latent vector
constexpr int kLogits = 4;             // tiles' logits in tensor memory
constexpr int kLoaders = 2;            // loading warps
constexpr int kThreads = 32 * (10 + kLoaders);
constexpr float kLift = 6.0f;          // a new reference: so far below the row's maximum
constexpr float kRedo = 32768.0f;      // a weight above it asks for one
constexpr int kFewSeqs = 48;           // sequences whose items are counted a warp each
// What an item takes beside its key tiles (queries in, first products, rows out), in tiles.
// (At 2, 3 and 5 the 24 ragged sequences took 98, 96 and 98 us.)
constexpr int kItemCost = 3;
constexpr int kSmemTop = 232448;       // shared memory a CTA can have

struct LatentDev : AttnArgs {
    int tops;                   // R / 128
    int rope_steps;             // 16-channel steps of the rotated part
    int heads, groups, tokens;  // an item: heads (of so many groups), tokens
    int ring;                   // tiles in shared memory
    float *acc;                 // partial outputs [2 * CTAs][NR][R]
    float2 *ml;                 // their references and sums [2 * CTAs][NR]
    int4 *join;                 // [CTAs]: what join_kernel joins
};

// ---------------------------------------------------------------- items ---
struct Item {
    int i0, cnt;    // tokens of the sequence's new ones
    int lo, hi;     // keys [lo, hi) that any of them sees
    int j0, tiles;  // key tiles: one at least, so that rows that see nothing are written
};
__device__ __forceinline__ Item item_of(const LatentDev &a, const Seq &s, int tile) {
    Item it;
    it.i0 = tile * a.tokens;
    it.cnt = min(a.tokens, s.n - it.i0);
    const int p0 = s.first + it.i0;
    it.hi = max(p0 + it.cnt, 0);
    it.lo = a.window > 0 ? min(max(p0 - a.window + 1, 0), it.hi) : 0;
    it.j0 = it.lo / kKeys;
    it.tiles = max((it.hi + kKeys - 1) / kKeys - it.j0, 1);
    return it;
}

// A CTA's walk along the line of items, the same in every role and in every CTA of a team.
// The line counts an item as kItemCost units and then its tiles.
struct Walk {
    int b, tile;
    int off;    // units of the item that lie before
    int k;      // segments taken
    long left;  // units
    Seq s;
};
struct Segment {
    Item it;
    int b, s0, p0;
    int j0, j1;         // key tiles
    bool starts, ends;  // whether it holds its item's first and last tile
    int k;
};
__device__ __forceinline__ bool next_segment(const LatentDev &a, Walk &w, Segment &g) {
    if (w.left <= 0) return false;
    g.it = item_of(a, w.s, w.tile);
    const int units = g.it.tiles + kItemCost;
    const int take = static_cast<int>(min(static_cast<long>(units - w.off), w.left));
    // the item's tiles are another CTA's: it begins with its first tile
    if (w.off + take <= kItemCost) return false;
    g.b = w.b;
    g.s0 = w.s.s0;
    g.p0 = w.s.first + g.it.i0;
    g.j0 = g.it.j0 + max(w.off - kItemCost, 0);
    g.j1 = g.it.j0 + w.off + take - kItemCost;
    g.starts = w.off <= kItemCost;
    g.ends = w.off + take == units;
    g.k = w.k++;
    w.left -= take;
    w.off = 0;
    if (w.left > 0) {
        if ((w.tile + 1) * a.tokens < w.s.n) {
            ++w.tile;
        } else {
            w.tile = 0;
            do {
                if (++w.b >= a.c.batch) {  // the line has no more items
                    w.left = 0;
                    break;
                }
                w.s = seq_of(a, w.b, false);
            } while (w.s.n == 0);
        }
    }
    return true;
}

// 16 lanes' N columns of the calling warp's quarter: v[4 i + e] is lane l / 4 (e < 2) or
// l / 4 + 8, column 8 i + 2 (l % 4) + e % 2.
template <int N>
__device__ __forceinline__ void tmem_ld_rows(uint32_t addr, float (&v)[N / 2]) {
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    if constexpr (N == 8) {
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(addr));
    } else {
#pragma unroll
        for (int i = 0; i < N / 2; i += 8)
            asm volatile(
                "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                : "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]),
                  "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
                : "r"(addr + 2 * i));
    }
}
// After tmem_wait_ld: no use of the loaded values moves above this point.
template <int N>
__device__ __forceinline__ void pin_rows(float (&v)[N / 2]) {
#pragma unroll
    for (int i = 0; i < N / 2; i += 4)
        asm volatile("" : "+f"(v[i]), "+f"(v[i + 1]), "+f"(v[i + 2]), "+f"(v[i + 3]));
}

// Barriers of the 256 softmax threads; the second tells whether any said yes.
__device__ __forceinline__ void meet() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ bool any_says(bool mine) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
        "bar.red.or.pred p, 1, 256, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(mine))
        : "memory");
    return r != 0;
}

// What stands behind the tiles in shared memory.
struct Small {
    uint64_t q_full, q_empty, full[kMaxRing][kMaxTops + 1], empty[kMaxRing][kMaxTops + 1],
        s_full[kLogits], p_full[kLogits], o_done[2], done;
    uint32_t tmem_slot;
    int abort_flag, found_seq;
    uint32_t dead_groups[16];  // per key tile: its 16-key groups on bad pages
    alignas(16) float m[64];  // rows' references,
    union {
        alignas(16) float base[64];     // less or 0,
        int row_at[64];                 // (at a segment's end: token * 65536 + head, -1: none)
    };
    alignas(16) float f[64];            // and the factor to a new one
    union {
        alignas(16) float red[4][64];
        struct {
            long seq_units[kFewSeqs], scan_total[kThreads / 32], found_rest;
            Walk start;
        };
    };
};
static_assert(sizeof(Small) <= 3 * 1024, "two tiles of 576 channels and 64 rows leave no more");
static_assert(offsetof(Small, base) % 8 == 0, "read by pairs");

template <int NR>
struct LatentShape {
    static constexpr int kP = NR == 64 ? 1 : 2;  // buffers of weights, 64 keys of 128 bytes
    static constexpr uint32_t kColumns = NR == 64 ? 512 : NR == 32 ? 256 : 128;
};

template <bool BF16, int NR>
__global__ void __launch_bounds__(kThreads, 1)
latent_kernel(const __grid_constant__ LatentDev a, const __grid_constant__ CUtensorMap q_map,
              const __grid_constant__ CUtensorMap k_map) {
    using Sh = LatentShape<NR>;
    constexpr int kQChunk = NR * 128;  // 64 channels of the rows
    constexpr uint32_t kO = kLogits * NR;  // columns of O

    extern __shared__ __align__(1024) uint8_t smem[];
    const int parts = a.tops + 1;      // of a row: the rotated part, then 128 channels each
    const int tile_bytes = a.tops * kPair + kHalf;
    uint8_t *q_smem = smem;            // the rotated part's chunk first
    uint8_t *p_smem = q_smem + (2 * a.tops + 1) * kQChunk;
    uint8_t *ring = p_smem + Sh::kP * kHalf;
    Small &sm = *reinterpret_cast<Small *>(ring + a.ring * tile_bytes);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (smem_addr(smem) & 1023) {      // (the launch asks for no other shared memory)
        if (tid == 0) report_status(a.c.dev_status, KVD_ERR_CUDA);
        return;
    }
    if (warp == 8) tmem_alloc(&sm.tmem_slot, Sh::kColumns);
    if (tid == 0) {
        mbar_init(&sm.q_full, 1);
        mbar_init(&sm.q_empty, 1);
        for (int i = 0; i < a.ring; ++i)
            for (int p = 0; p < parts; ++p) {
                mbar_init(&sm.full[i][p], 1);
                mbar_init(&sm.empty[i][p], 1);
            }
        for (int i = 0; i < kLogits; ++i) {
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.p_full[i], 8);
        }
        for (int i = 0; i < 2; ++i) mbar_init(&sm.o_done[i], 1);
        mbar_init(&sm.done, 2);
        fence_barrier_init();
        sm.abort_flag = 0;
        sm.start.left = 0;
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    pdl_wait();
    pdl_launch_dependents();

    // ---- this CTA's piece of the line of items
    // of a sequence: a warp's lanes take a run of tokens each
    auto units_of = [&](const Seq &s) -> long {
        long n = 0;
#pragma unroll 1
        for (int t = lane; t * a.tokens < s.n; t += 32) n += item_of(a, s, t).tiles + kItemCost;
#pragma unroll
        for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
        return n;
    };
    constexpr int kAlone = 16;  // items that a lane counts by itself
    auto cost_of = [&](int b, bool report) -> long {
        Seq s = {};
        if (b < a.c.batch) s = seq_of(a, b, report);
        const bool many = s.n > kAlone * a.tokens;
        long n = 0;
#pragma unroll 1
        for (int t = 0; !many && t * a.tokens < s.n; ++t) n += item_of(a, s, t).tiles + kItemCost;
        uint32_t more = __ballot_sync(0xffffffffu, many);
#pragma unroll 1
        for (; more; more &= more - 1) {
            const int l = __ffs(more) - 1;
            const long u = units_of(seq_of(a, b - lane + l, false));
            if (lane == l) n = u;
        }
        return n;
    };
    auto scan = [&](long cost, long &before) -> long {  // exclusive prefix, and the sum
        long v = cost;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        if (lane == 31) sm.scan_total[warp] = v;
        __syncthreads();
        long sum = 0;
        before = v - cost;
        for (int i = 0; i < kThreads / 32; ++i) {
            if (i < warp) before += sm.scan_total[i];
            sum += sm.scan_total[i];
        }
        __syncthreads();
        return sum;
    };
    // unit r of sequence b's: the run of tokens, 32 at a time
    auto walk_from = [&](int b, long r) -> Walk {
        Walk w;
        w.b = b;
        w.s = seq_of(a, b, false);
#pragma unroll 1
        for (int t0 = 0;; t0 += 32) {
            const int t = t0 + lane;
            const int n = t * a.tokens < w.s.n ? item_of(a, w.s, t).tiles + kItemCost : 0;
            long upto = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long u = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += u;
            }
            const uint32_t in = __ballot_sync(0xffffffffu, r < upto);
            if (in || t0 * a.tokens >= w.s.n) {
                const int l = in ? __ffs(in) - 1 : 0;
                w.tile = t0 + l;
                w.off = static_cast<int>(r - __shfl_sync(0xffffffffu, upto - n, l));
                break;
            }
            r -= __shfl_sync(0xffffffffu, upto, 31);
        }
        w.k = 0;
        return w;
    };
    const int group = blockIdx.x % a.groups, team = blockIdx.x / a.groups;
    const long most = gridDim.x / a.groups;
    long total = 0, share = 0, spare = 0, x0 = 0, x1 = 0;
    auto cut = [&](long c) { return c * share + min(c, spare); };  // where team c begins
    auto cut_line = [&] {  // this team's piece [x0, x1)
        const long per = max((total + most - 1) / most, static_cast<long>(a.min_tiles));
        const long teams = max(min(most, (total + per - 1) / per), 1l);
        share = total / teams;
        spare = total % teams;
        x0 = team < teams ? cut(team) : total;
        x1 = team < teams ? cut(team + 1) : total;
    };
    Walk w;
    w.left = 0;
    if (a.c.batch <= 32 && a.max_new <= kAlone * a.tokens) {
        // short: each warp finds it by itself, a lane a sequence
        const long cost = cost_of(lane, blockIdx.x == 0 && warp == 0);
        long upto = cost;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long u = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += u;
        }
        total = __shfl_sync(0xffffffffu, upto, 31);
        cut_line();
        if (x0 < x1) {
            const uint32_t in =
                __ballot_sync(0xffffffffu, upto - cost <= x0 && x0 < upto);
            const int l = __ffs(in) - 1;
            w = walk_from(l, x0 - __shfl_sync(0xffffffffu, upto - cost, l));
            w.left = x1 - x0;
        }
    } else {
        long before = 0, cost;
        if (a.c.batch <= kFewSeqs) {
#pragma unroll 1
            for (int b = warp; b < a.c.batch; b += kThreads / 32) {
                const long n = units_of(seq_of(a, b, blockIdx.x == 0));
                if (lane == 0) sm.seq_units[b] = n;
            }
            __syncthreads();
            cost = tid < a.c.batch ? sm.seq_units[tid] : 0;
        } else {
            cost = cost_of(tid, blockIdx.x == 0);
        }
        total = scan(cost, before);
        const bool one_pass = a.c.batch <= kThreads;
#pragma unroll 1
        for (int b0 = kThreads; b0 < a.c.batch; b0 += kThreads) {
            long skip;
            total += scan(cost_of(b0 + tid, blockIdx.x == 0), skip);
        }
        cut_line();
        if (x0 < x1) {
            long base = 0;
#pragma unroll 1
            for (int b0 = 0; b0 < a.c.batch; b0 += kThreads) {
                if (!one_pass) {
                    cost = cost_of(b0 + tid, false);
                    const long sum = scan(cost, before);
                    before += base;
                    base += sum;
                }
                if (before <= x0 && x0 < before + cost) {
                    sm.found_seq = b0 + tid;
                    sm.found_rest = x0 - before;
                }
            }
            __syncthreads();
            if (warp == 0) {  // the run of tokens, 32 at a time
                Walk w = walk_from(sm.found_seq, sm.found_rest);
                w.left = x1 - x0;
                if (lane == 0) sm.start = w;
            }
        }
        __syncthreads();
        w = sm.start;
        __syncthreads();  // `start` has been read: its memory is the softmax's
    }
    const uint32_t tmem = sm.tmem_slot;
    Segment g;
    volatile int *abort = &sm.abort_flag;
    auto fail = [&] {
        *abort = 1;
        report_status(a.c.dev_status, KVD_ERR_TIMEOUT);
    };
    bool ok = true;

    if (warp >= 10) {
        // ------------------------------------------------------------ loads ---
        // rows that other items read too stay in the L2
        const bool shared = a.groups > 1 || a.max_new > a.tokens;
        const uint64_t policy = shared ? l2_policy_evict_last() : l2_policy_evict_first();
        const int boxes = kKeys / a.box, ps = a.c.page_size;
        const int per_read = 32 / boxes;  // tiles whose rows one read of the page table gives
        // Lane l of warp w loads part w + kLoaders l of each tile: the rotated part (0), or the
        // channels [128 (p - 1), 128 p)
        const bool first_warp = warp == 10;     // and queries
        const int part = warp - 10 + kLoaders * lane;
        const bool loads = part < parts;
        const int my_part = loads ? part : 0;
        const int my_x = part == 0 ? a.tops * 128 : (part - 1) * 128;
        const int my_at = part == 0 ? a.tops * kPair : (part - 1) * kPair;
        uint32_t n = 0, mine = 0, queries = 0;  // tiles, this lane's loads of them, of queries
        uint32_t st = 0, round = 0;
        int4 rec = make_int4(0, 0, 0, 0);
#pragma unroll 1
        while (ok && next_segment(a, w, g)) {
            if (first_warp) {
                if (queries > 0 && !(ok = wait_for(&sm.q_empty, (queries - 1) & 1, abort))) break;
                ++queries;
                if (lane == 0)
                    mbar_arrive_expect_tx(&sm.q_full, (2 * a.tops + 1) * a.heads * a.tokens * 128);
                __syncwarp();
            }
            if (first_warp && lane <= 2 * a.tops)
                tma_load_4d(q_smem + lane * kQChunk, &q_map, lane == 0 ? a.tops * 128 : (lane - 1) * 64,
                            group * a.heads, 0, g.s0 + g.it.i0, &sm.q_full);
            // the cache rows of the boxes of tiles j, j + 1, .., a lane a box: dead_row
            // where none is needed, -1 on a bad page
            auto rows_of = [&](int j) -> int {
                const int t0 = (j + lane / boxes) * kKeys + lane % boxes * a.box;
                if (t0 >= g.j1 * kKeys || t0 >= g.it.hi || t0 + a.box <= g.it.lo) return a.dead_row;
                const int col = t0 / ps;
                const int page = checked_page(a.c, g.b, col);
                return page < 0 ? -1 : page * ps + (t0 - col * ps);
            };
            int rows = 0, rows_next = rows_of(g.j0);
#pragma unroll 1
            for (int j = g.j0; j < g.j1; ++j) {
                const int in = (j - g.j0) % per_read;
                if (in == 0) {
                    rows = rows_next;
                    rows_next = rows_of(j + per_read);
                }
                int row[4];
                uint32_t bad = 0;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    row[x] = __shfl_sync(0xffffffffu, rows, in * boxes + min(x, boxes - 1));
                    if (row[x] < 0) {
                        row[x] = a.dead_row;
                        if (x < boxes) bad |= ((1u << (a.box / 16)) - 1) << (x * (a.box / 16));
                    }
                }
                if (first_warp && lane == 0) sm.dead_groups[n & 15] = bad;
                __syncwarp();
                // each part as soon as its place is free (a fresh barrier's is)
                uint64_t *full = &sm.full[st][my_part];
                uint8_t *dst = ring + st * tile_bytes + my_at;
                ok = each_when(loads, &sm.empty[st][my_part], ~round & 1, abort, [&] {
                    mbar_arrive_expect_tx(full, part == 0 ? kHalf : kPair);
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        if (x < boxes) {
                            tma_load_2d(dst + x * a.box * 128, &k_map, my_x, row[x], full, policy);
                            if (part > 0)
                                tma_load_2d(dst + kHalf + x * a.box * 128, &k_map, my_x + 64, row[x],
                                            full, policy);
                        }
                    ++mine;
                });
                if (!ok) break;
                ++n;
                if (++st == static_cast<uint32_t>(a.ring)) {
                    st = 0;
                    ++round;
                }
            }
            if (ok && g.starts && !g.ends) {
                // the item goes on in the next teams: leave word for join_kernel
                const long rest = g.it.j0 + g.it.tiles - g.j1;  // tiles, and units
                int pieces = 1;
                while (cut(team + pieces + 1) - x1 < rest) ++pieces;
                rec = make_int4(pieces + 1, g.k == 0 ? 0 : 1, g.s0 + g.it.i0, g.it.cnt);
            }
        }
        if (!ok) fail();
        if (first_warp && lane == 0) {
            a.join[blockIdx.x] = rec;
        }
        tmem_fence_before();
        __syncthreads();  // all roles are done, and know whether a wait ran out
        if (*abort) {
            // nothing may land in shared memory after the CTA has gone
            volatile int none = 0;
            bool landed = true;  // after one wait that runs out all has had the time to land
            for (uint32_t i = 0; loads && landed && i < static_cast<uint32_t>(a.ring); ++i) {
                const uint32_t fills = (mine + a.ring - 1 - i) / a.ring;
                if (fills > 0) landed = mbar_wait(&sm.full[i][part], (fills - 1) & 1, &none);
            }
            __syncwarp();
            if (queries > 0) mbar_wait(&sm.q_full, (queries - 1) & 1, &none);
        }
        return;
    } else if (warp == 8) {
        // -------------------------------------------------- products S^T = K Q^T ---
        constexpr uint32_t kIdS = mma_idesc(BF16, kKeys, NR, false);
        const uint32_t ring_addr = smem_addr(ring);
        const uint32_t q = warp_uniform(desc_low(smem_addr(q_smem), 16));
        const uint32_t tmem_u = warp_uniform(tmem);
        uint32_t n = 0, st = 0, round = 0, queries = 0;
#pragma unroll 1
        while (ok && next_segment(a, w, g)) {
            if (!(ok = wait_for(&sm.q_full, queries & 1, abort))) break;
            ++queries;
#pragma unroll 1
            for (int j = g.j0; ok && j < g.j1; ++j, ++n) {
                const uint32_t b = n % kLogits;
                // the logits that were there have been read
                if (n >= kLogits && !(ok = wait_for(&sm.p_full[b], (n / kLogits - 1) & 1, abort)))
                    break;
                tmem_fence_after();
                const uint32_t s_at = warp_uniform(tmem_u + b * NR);
                const uint32_t k = warp_uniform(desc_low(ring_addr + st * tile_bytes, 16));
                const uint32_t k_rope = warp_uniform(k + a.tops * (kPair / 16));
#pragma unroll
                for (int p = 0; p <= kMaxTops; ++p) {
                    if (p > a.tops) break;
                    if (!(ok = wait_for(&sm.full[st][p], round & 1, abort))) break;
                    if (elect_one()) {
                        if (p == 0) {
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                if (x < a.rope_steps)
                                    mma_ss(s_at, smem_desc(k_rope + 2 * x), smem_desc(q + 2 * x), kIdS,
                                           x > 0);
                            mma_commit(&sm.empty[st][0]);
                        } else {
#pragma unroll
                            for (int x = 0; x < 8; ++x)
                                mma_ss(s_at,
                                       smem_desc(k + ((p - 1) * kPair + x / 4 * kHalf) / 16 + x % 4 * 2),
                                       smem_desc(q + (2 * p - 1 + x / 4) * (kQChunk / 16) + x % 4 * 2),
                                       kIdS, 1);
                            if (p == a.tops) {
                                mma_commit(&sm.s_full[b]);
                                if (j + 1 == g.j1) mma_commit(&sm.q_empty);
                            }
                        }
                    }
                    __syncwarp();
                }
                if (++st == static_cast<uint32_t>(a.ring)) {
                    st = 0;
                    ++round;
                }
            }
        }
        if (!ok) fail();
        // every product and every barrier arrival is done before the CTA goes
        if (elect_one()) mma_commit(&sm.done);
        __syncwarp();
        volatile int none = 0;
        if (!mbar_wait(&sm.done, 0, &none)) fail();
    } else if (warp == 9) {
        // ---------------------------------------------- products O^T += V^T P^T ---
        constexpr uint32_t kIdO = mma_idesc(BF16, 128, NR, true, true);
        const uint32_t ring_addr = smem_addr(ring);
        const uint32_t tmem_u = warp_uniform(tmem);
        uint32_t n = 0, st = 0, round = 0;
#pragma unroll 1
        while (ok && next_segment(a, w, g)) {
#pragma unroll 1
            for (int j = g.j0; j < g.j1; ++j, ++n) {
                const uint32_t b = n & 1;
                if (!(ok = wait_for(&sm.p_full[n % kLogits], (n / kLogits) & 1, abort))) break;
                // (they have landed: the logits come from them)
                if (!(ok = each_when(lane > 0 && lane < parts, &sm.full[st][min(lane, a.tops)],
                                     round & 1, abort, [] {})))
                    break;
                tmem_fence_after();
                const uint32_t p = warp_uniform(
                    desc_low(smem_addr(p_smem) + (Sh::kP == 2 ? b * kHalf : 0), kHalf));
                const uint32_t add = warp_uniform(j > g.j0);
                const uint32_t v = warp_uniform(desc_low(ring_addr + st * tile_bytes, kHalf));
                if (elect_one()) {
#pragma unroll
                    for (int m = 0; m < kMaxTops; ++m) {
                        if (m >= a.tops) break;
#pragma unroll
                        for (int x = 0; x < kKeys / 16; ++x)
                            mma_ss(tmem_u + kO + m * NR, smem_desc(v + (m * kPair + x * 2048) / 16),
                                   smem_desc(p + x * (2048 / 16)), kIdO, x > 0 ? 1 : add);
                        mma_commit(&sm.empty[st][1 + m]);
                    }
                    mma_commit(&sm.o_done[b]);
                }
                __syncwarp();
                if (++st == static_cast<uint32_t>(a.ring)) {
                    st = 0;
                    ++round;
                }
            }
        }
        if (!ok) fail();
        if (elect_one()) mma_commit(&sm.done);
        __syncwarp();
        volatile int none = 0;
        if (!mbar_wait(&sm.done, 0, &none)) fail();
    } else {
        // ------------------------------------------------------------ softmax ---
        constexpr int kV = NR / 4;   // logits a thread: 4 for each 8 of the half's rows
        const int quarter = warp & 3, half = warp >> 2;
        const uint32_t lanes = tmem + (quarter << 21);
        const int key0 = quarter * 16 + lane / 4, col0 = half * (NR / 2) + 2 * (lane & 3);
        const int R = a.tops * 128;
        const int my_tok = tid / a.heads, my_head = tid - my_tok * a.heads;  // of row `tid`
        uint32_t n = 0, st = 0;
        // These warps meet at barriers of the hardware, which have no limit: so none
        // leaves its loops before the others, and a wait that ran out only makes the
        // waits behind it pass.
        auto wait = [&](uint64_t *b, uint32_t parity) {
            if (ok) ok = wait_for(b, parity, abort);
        };
#pragma unroll 1
        while (next_segment(a, w, g)) {
            const int heads = min(a.heads, a.G - group * a.heads);
            // keys that every row sees
            const int all_lo = a.window > 0 ? max(g.p0 + g.it.cnt - a.window, 0) : 0;
            const int all_hi = max(g.p0 + 1, 0);
            const bool live = my_tok < g.it.cnt && my_head < heads;
            float l[kV / 2];
#pragma unroll
            for (int i = 0; i < kV / 2; ++i) l[i] = 0.0f;
            bool open = true;  // a row has seen no key yet, and so has no reference
#pragma unroll 1
            for (int j = g.j0; j < g.j1; ++j, ++n) {
                const uint32_t s_at = lanes + n % kLogits * NR + half * (NR / 2);
                wait(&sm.s_full[n % kLogits], (n / kLogits) & 1);
                const bool bad = sm.dead_groups[n & 15] >> quarter & 1;
                // the rows [r0, r1) that see each of the two keys
                int r0[2] = {0, 0}, r1[2] = {NR, NR};
                const bool edge = j * kKeys < all_lo || (j + 1) * kKeys > all_hi || bad;
                if (edge) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int t = j * kKeys + key0 + 8 * e;
                        r1[e] = 0;
                        if (t >= g.it.lo && t < g.it.hi && !bad) {
                            const int first = max(t - g.p0, 0);
                            int last = g.it.cnt - 1;
                            if (a.window > 0) last = min(last, t + a.window - 1 - g.p0);
                            if (first <= last) {
                                r0[e] = first * a.heads;
                                r1[e] = (last + 1) * a.heads;
                            }
                        }
                    }
                }
                tmem_fence_after();
                auto hidden = [&](int i) {
                    const int r = i / 4 * 8 + col0 + (i & 1), e = i >> 1 & 1;
                    return r < r0[e] || r >= r1[e];
                };
                bool fix = open;
                float p[kV];
#pragma unroll 1
                for (;;) {
                    float s[kV];
                    tmem_ld_rows<NR / 2>(s_at, s);
                    tmem_wait_ld();
                    pin_rows<NR / 2>(s);
                    if (edge)
#pragma unroll
                        for (int i = 0; i < kV; ++i)
                            if (hidden(i)) s[i] = -INFINITY;
                    if (fix) {
                        // each row's maximum, over the warp's keys, then over all
#pragma unroll
                        for (int i = 0; i < kV; i += 4)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float t = fmaxf(s[i + e], s[i + 2 + e]);
#pragma unroll
                                for (int o = 4; o < 32; o <<= 1)
                                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
                                if (lane < 4) sm.red[quarter][i / 4 * 8 + col0 + e] = t;
                            }
                        // O as it stands is complete
                        if (j > g.j0) wait(&sm.o_done[(n - 1) & 1], ((n - 1) >> 1) & 1);
                        meet();
                        bool none = false;
                        if (tid < NR) {
                            const float top = fmaxf(fmaxf(sm.red[0][tid], sm.red[1][tid]),
                                                    fmaxf(sm.red[2][tid], sm.red[3][tid]));
                            const float m = j == g.j0 ? -INFINITY : sm.m[tid];
                            const float mn = fmaxf(m, top * a.scale_log2 - kLift);
                            sm.f[tid] =
                                m == -INFINITY || mn == -INFINITY ? 1.0f : exp2_approx(m - mn);
                            sm.m[tid] = mn;
                            none = live && mn == -INFINITY;
                            // rows that are none (another sequence's queries may stand
                            // there): no weights, and no say in the votes
                            sm.base[tid] = !live ? -INFINITY : mn == -INFINITY ? 0.0f : -mn;
                        }
                        open = any_says(none);
#pragma unroll
                        for (int i = 0; i < kV / 2; ++i) l[i] *= sm.f[i / 2 * 8 + col0 + (i & 1)];
                        if (j > g.j0) {
                            tmem_fence_after();
#pragma unroll 1
                            for (int i = 16 * half; i < a.tops * NR; i += 32) {
                                float o[16];
                                tmem_ld16(lanes + kO + i, o);
                                tmem_wait_ld();
                                pin16(o);
#pragma unroll
                                for (int r = 0; r < 16; ++r) o[r] *= sm.f[i % NR + r];
                                tmem_st16(lanes + kO + i, reinterpret_cast<uint32_t *>(o));
                            }
                            tmem_wait_st();
                            tmem_fence_before();
                        }
                    }
                    const float2 k2 = make_float2(a.scale_log2, a.scale_log2);
                    float top = 0.0f;
#pragma unroll
                    for (int i = 0; i < kV; i += 4) {
                        const float2 base =
                            *reinterpret_cast<const float2 *>(&sm.base[i / 4 * 8 + col0]);
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            const float2 x = __ffma2_rn(make_float2(s[i + e], s[i + e + 1]), k2, base);
                            p[i + e] = exp2_approx(x.x);
                            p[i + e + 1] = exp2_approx(x.y);
                        }
                    }
                    if (edge)  // (a row without a reference yet, or -infinity less infinity)
#pragma unroll
                        for (int i = 0; i < kV; ++i)
                            if (hidden(i)) p[i] = 0.0f;
#pragma unroll
                    for (int i = 0; i < kV; i += 2) top = fmax3(top, p[i], p[i + 1]);
                    if (fix) break;  // no weight passes 2^kLift
                    if (!any_says(top > kRedo)) break;
                    fix = true;
                }
                // P^T's buffer has been read
                if (n >= Sh::kP) wait(&sm.o_done[(n - Sh::kP) & 1], ((n - Sh::kP) >> 1) & 1);
                const int from = g.it.lo - j * kKeys, to = g.it.hi - j * kKeys;
                if (from > 0 || to < kKeys) {
                    // rows that no token sees may hold NaN: clear them (they have landed, and
                    // the logits are done)
                    uint8_t *vs = ring + st * tile_bytes + (tid >> 3 & 1) * kHalf + (tid & 7) * 16;
#pragma unroll 1
                    for (int r = tid >> 4; r < kKeys; r += 16)
                        if (r < from || r >= to)
                            for (int x = 0; x < a.tops; ++x)
                                *reinterpret_cast<uint4 *>(vs + x * kPair + r * 128) =
                                    make_uint4(0, 0, 0, 0);
                }
                // the weights, and P^T: a key's rows in 128 swizzled bytes
                uint8_t *dst = p_smem + (Sh::kP == 2 ? (n & 1) * kHalf : 0) + key0 * 128 + (lane & 3) * 4;
#pragma unroll
                for (int i = 0; i < kV; i += 4) {
                    l[i / 2] += p[i] + p[i + 2];
                    l[i / 2 + 1] += p[i + 1] + p[i + 3];
                    const int at = ((i / 4 + half * (NR / 16)) ^ (key0 & 7)) * 16;  // (key0 + 8 has the same low bits)
                    *reinterpret_cast<uint32_t *>(dst + at) = pack2<BF16>(p[i], p[i + 1]);
                    *reinterpret_cast<uint32_t *>(dst + 1024 + at) = pack2<BF16>(p[i + 2], p[i + 3]);
                }
                fence_proxy_async();
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.p_full[n % kLogits]);
                if (++st == static_cast<uint32_t>(a.ring)) st = 0;
            }
            // ---- the segment's sums
            meet();  // the last references have been read
#pragma unroll
            for (int i = 0; i < kV / 2; ++i) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
                if (lane < 4) sm.red[quarter][i / 2 * 8 + col0 + (i & 1)] = l[i];
            }
            wait(&sm.o_done[(n - 1) & 1], ((n - 1) >> 1) & 1);
            tmem_fence_after();
            meet();
            const bool whole = g.starts && g.ends;
            const uint32_t slot = 2 * blockIdx.x + (g.k == 0 ? 0 : 1);
            if (tid < NR) {
                const float sum = (sm.red[0][tid] + sm.red[1][tid]) + (sm.red[2][tid] + sm.red[3][tid]);
                const float m = sm.m[tid];
                sm.f[tid] = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
                const int h = group * a.heads + my_head;
                sm.row_at[tid] = live ? my_tok << 16 | h : -1;
                if (live) {
                    if (!whole)
                        a.ml[slot * NR + tid] = make_float2(m, sum);
                    else if (a.lse)
                        a.lse[static_cast<int64_t>(g.s0 + g.it.i0 + my_tok) * a.G + h] = lse_of(m, sum);
                }
            }
            meet();
            const int rows = g.it.cnt * a.heads;
            // A thread holds a channel of 16 rows at a time.
#pragma unroll 1
            for (int x = half; x < a.tops * (NR / 16); x += 2) {
                const int m = x / (NR / 16), i = x % (NR / 16) * 16;
                if (i >= rows) continue;
                const int channel = m * 128 + quarter * 32 + lane;
                float o[16];
                tmem_ld16(lanes + kO + m * NR + i, o);
                tmem_wait_ld();
                pin16(o);
                if (whole) {
                    uint16_t *out = a.out + static_cast<int64_t>(g.s0 + g.it.i0) * a.out_stride +
                                    (channel & ~1);
                    // even lanes take two channels of the even rows, odd lanes of the odd ones
                    const bool odd = lane & 1;
#pragma unroll
                    for (int r = 0; r < 16; r += 2) {
                        const float f0 = sm.f[i + r], f1 = sm.f[i + r + 1];
                        const float o0 = f0 != 0.0f ? o[r] * f0 : 0.0f;
                        const float o1 = f1 != 0.0f ? o[r + 1] * f1 : 0.0f;
                        const float other = __shfl_xor_sync(0xffffffffu, odd ? o0 : o1, 1);
                        const int to = sm.row_at[i + r + odd];
                        if (to >= 0)
                            *reinterpret_cast<uint32_t *>(out + (to >> 16) * a.out_stride +
                                                          (to & 0xffff) * R) =
                                odd ? pack2<BF16>(other, o1) : pack2<BF16>(o0, other);
                    }
                } else {
                    float *to = a.acc + (static_cast<int64_t>(slot) * NR + i) * R + channel;
#pragma unroll
                    for (int r = 0; r < 16; ++r, to += R)
                        if (i + r < rows) *to = o[r];
                }
            }
            tmem_fence_before();
            meet();  // the next segment's references go where these stood
        }
        if (!ok) fail();
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == 8) {
        tmem_fence_after();
        tmem_free(tmem, Sh::kColumns);
    }
}

// Joins the items that a cut between CTAs divided: the rows of all such items stand in one
// line (record c: the item whose first piece is CTA c's last segment and goes on in its
// group's CTA of the teams after it).
//   out = sum_i 2^(m_i - m) acc_i / sum_i 2^(m_i - m) l_i
// A warp takes PARTS times 128 channels of a row, the reads of AT pieces under way together.
constexpr int kMaxCtas = 256;
constexpr int kJoinThreads = 128;
template <bool BF16, int NR, int PARTS, int AT>
__device__ __forceinline__ void join_rows(const LatentDev &a, const int *before, const int4 *recs, int w,
                                          int warps, int lane) {
    const int R = a.tops * 128, units = PARTS == 1 ? a.tops : 1;
#pragma unroll 1
    for (; w < before[kMaxCtas] * units; w += warps) {
        const int u = w / units, part = w - u * units;
        int c = 0;  // the last record that begins at or before u
#pragma unroll
        for (int step = kMaxCtas / 2; step > 0; step >>= 1)
            if (before[c + step] <= u) c += step;
        const int r = u - before[c];
        const int4 rec = recs[c];  // pieces, whether the first is its CTA's second segment, token, tokens
        const int group = c % a.groups;
        const int tok = r / a.heads, h = group * a.heads + r - tok * a.heads;
        if (h >= a.G) continue;
        // piece i is CTA c + i * groups's first segment, the first piece maybe its second
        auto slot_of = [&](int i) {
            return static_cast<size_t>(2 * (c + i * a.groups) + (i == 0 ? rec.y : 0));
        };
        const float *acc = a.acc + static_cast<size_t>(r) * R + part * 128 + lane * 4;
        float4 v[AT][PARTS];
        auto read = [&](int i0, int n) {  // pieces i0 .. i0 + n, AT at most
#pragma unroll
            for (int x = 0; x < AT; ++x)
#pragma unroll
                for (int p = 0; p < PARTS; ++p)
                    if (x < n && (PARTS == 1 || p < a.tops))
                        v[x][p] = *reinterpret_cast<const float4 *>(acc + slot_of(i0 + x) * NR * R + 128 * p);
        };
        read(0, rec.x);  // (beside the references)
        float m = -INFINITY, l = 0.0f;
        for (int i = lane; i < rec.x; i += 32) m = fmaxf(m, a.ml[slot_of(i) * NR + r].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        float4 o[PARTS];
#pragma unroll
        for (int p = 0; p < PARTS; ++p) o[p] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
        for (int i0 = 0; i0 < rec.x; i0 += 32) {
            float f = 0.0f;  // of piece i0 + lane
            if (i0 + lane < rec.x) {
                const float2 ml = a.ml[slot_of(i0 + lane) * NR + r];
                f = ml.x == -INFINITY ? 0.0f : exp2_approx(ml.x - m);
                l = fmaf(f, ml.y, l);  // a sum that is NaN stays one where f is 0
            }
            const int n = min(32, rec.x - i0);
#pragma unroll 1
            for (int i = 0; i < n; i += AT) {
                if (i0 + i > 0) read(i0 + i, n - i);
#pragma unroll
                for (int x = 0; x < AT; ++x) {
                    const float g = __shfl_sync(0xffffffffu, f, (i + x) & 31);
                    if (i + x < n && g != 0.0f)
#pragma unroll
                        for (int p = 0; p < PARTS; ++p) {
                            o[p].x = fmaf(g, v[x][p].x, o[p].x);
                            o[p].y = fmaf(g, v[x][p].y, o[p].y);
                            o[p].z = fmaf(g, v[x][p].z, o[p].z);
                            o[p].w = fmaf(g, v[x][p].w, o[p].w);
                        }
                }
            }
        }
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
        const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
        const int64_t token = rec.z + tok;
        if (a.lse && lane == 0 && part == 0) a.lse[token * a.G + h] = lse_of(m, l);
        uint16_t *out = a.out + token * a.out_stride + static_cast<int64_t>(h) * R + part * 128 + lane * 4;
#pragma unroll
        for (int p = 0; p < PARTS; ++p)
            if (PARTS == 1 || p < a.tops)
                *reinterpret_cast<uint2 *>(out + 128 * p) =
                    make_uint2(pack2<BF16>(o[p].x * inv, o[p].y * inv),
                               pack2<BF16>(o[p].z * inv, o[p].w * inv));
    }
}

template <bool BF16, int NR>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ LatentDev a, int ctas) {
    __shared__ int before[kMaxCtas + 1];  // rows of the records before
    __shared__ int4 recs[kMaxCtas];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_launch_dependents();
    if (warp == 0) {
        constexpr int kEach = kMaxCtas / 32;
        int n[kEach], sum = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int c = lane * kEach + i;
            int4 rec = make_int4(0, 0, 0, 0);
            if (c < ctas) rec = a.join[c];
            recs[c] = rec;
            n[i] = rec.x ? rec.w * a.heads : 0;
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) sum += n[i];
        int upto = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += u;
        }
        upto -= sum;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            before[lane * kEach + i] = upto;
            upto += n[i];
        }
        if (lane == 31) before[kMaxCtas] = upto;
    }
    __syncthreads();
    // A warp a row, or where there are few rows 128 channels of one: 128 rows of 38 pieces
    // 85.9 us with the attention, 90.9 the other way; 4096 rows of 3 or 4 pieces 110.3 and 120.7.
    const int warps = gridDim.x * (kJoinThreads / 32);
    const int w = blockIdx.x * (kJoinThreads / 32) + warp;
    if (before[kMaxCtas] * a.tops <= warps)
        join_rows<BF16, NR, 1, 8>(a, before, recs, w, warps, lane);
    else
        join_rows<BF16, NR, kMaxTops, 3>(a, before, recs, w, warps, lane);
}

// ----------------------------------------------------------------- launch ---
struct Plan {
    int ctas, heads, groups, tokens, nr;
    size_t ml, acc, total;
};

Plan plan_of(int H, int rank, int max_new) {
    Plan w;
    w.ctas = device_sm_count() < kMaxCtas ? device_sm_count() : kMaxCtas;
    w.groups = (H + 63) / 64;
    w.heads = (H + w.groups - 1) / w.groups;
    w.tokens = 64 / w.heads < max_new ? 64 / w.heads : max_new;
    const int rows = w.heads * w.tokens;
    // Fewer rows take less of shared memory's rate: one token of 16 heads over 4 sequences of
    // 100,000 84 us with 16, 85.5 with 32, 92 with 64; of 32 heads 86 and 93.
    w.nr = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    w.ml = up(static_cast<size_t>(w.ctas) * sizeof(int4));
    // (of any max_new: 64 rows)
    w.acc = w.ml + up(static_cast<size_t>(w.ctas) * 2 * 64 * sizeof(float2));
    w.total = w.acc + up(static_cast<size_t>(w.ctas) * 2 * w.nr * rank * sizeof(float));
    return w;
}

template <bool BF16, int NR>
cudaError_t launch_rows(const PagedAttnArgs &p, int rank, const Plan &w, void *ws, cudaStream_t st) {
    using Sh = LatentShape<NR>;
    const kvd_paged_cache &c = p.c;
    LatentDev a = {};
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
    while (a.box < kKeys && c.page_size % (2 * a.box) == 0) a.box *= 2;
    const int64_t pool = static_cast<int64_t>(c.n_pages) * c.page_size;
    a.dead_row = static_cast<int>(pool);
    a.min_tiles = kItemCost + 1;  // an item's first CTA takes a tile
    a.tops = rank / 128;
    a.rope_steps = (c.head_dim - rank) / 16;
    a.heads = w.heads;
    a.groups = w.groups;
    a.tokens = w.tokens;
    const int fixed = (2 * a.tops + 1) * NR * 128 + Sh::kP * kHalf + static_cast<int>(sizeof(Small));
    const int tile = a.tops * kPair + kHalf;
    a.ring = (kSmemTop - fixed) / tile;
    if (a.ring > kMaxRing) a.ring = kMaxRing;
    const size_t smem = static_cast<size_t>(fixed) + static_cast<size_t>(a.ring) * tile;
    uint8_t *base = static_cast<uint8_t *>(ws);
    a.join = reinterpret_cast<int4 *>(base);
    a.ml = reinterpret_cast<float2 *>(base + w.ml);
    a.acc = reinterpret_cast<float *>(base + w.acc);

    CUtensorMap q_map, k_map;
    const cuuint64_t W = static_cast<cuuint64_t>(c.head_dim);
    const cuuint64_t qd[4] = {W, static_cast<cuuint64_t>(p.G), 1, static_cast<cuuint64_t>(p.n_tokens)};
    const cuuint64_t qs[3] = {W * 2, W * 2 * p.G, static_cast<cuuint64_t>(p.q_stride) * 2};
    const cuuint32_t qb[4] = {64, static_cast<cuuint32_t>(a.heads), 1, static_cast<cuuint32_t>(a.tokens)};
    const cuuint64_t kd[2] = {W, static_cast<cuuint64_t>(pool)};
    const cuuint64_t ks[1] = {W * 2};
    const cuuint32_t kb[2] = {64, static_cast<cuuint32_t>(a.box)};
    if (!make_map(&q_map, c.dtype, p.q, 4, qd, qs, qb) || !make_map(&k_map, c.dtype, c.k, 2, kd, ks, kb))
        return cudaErrorInvalidValue;
    auto *kernel = latent_kernel<BF16, NR>;
    cudaError_t e = prepare_kernel(reinterpret_cast<const void *>(kernel), kThreads, smem);
    if (e != cudaSuccess) return e;
    e = launch_ex(kernel, dim3(w.ctas), dim3(kThreads), smem, st, true, a, q_map, k_map);
    if (e != cudaSuccess) return e;
    return launch_ex(join_kernel<BF16, NR>, dim3(4 * w.ctas), dim3(kJoinThreads), 0, st, true, a, w.ctas);
}

template <bool BF16>
cudaError_t launch_type(const PagedAttnArgs &p, int rank, void *ws, cudaStream_t st) {
    const Plan w = plan_of(p.G, rank, p.max_new);
    if (w.nr == 16) return launch_rows<BF16, 16>(p, rank, w, ws, st);
    if (w.nr == 32) return launch_rows<BF16, 32>(p, rank, w, ws, st);
    return launch_rows<BF16, 64>(p, rank, w, ws, st);
}

}  // namespace

cudaError_t launch_latent_attn(const PagedAttnArgs &a, int rank, void *ws, cudaStream_t st) {
    return a.bf16 ? launch_type<true>(a, rank, ws, st) : launch_type<false>(a, rank, ws, st);
}

size_t latent_attn_ws(int H, int rank, int max_new) { return plan_of(H, rank, max_new).total; }

}  // namespace kvd
