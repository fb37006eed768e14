// paged_attn.cu -- attention of a ragged batch's new tokens over a paged cache.
//
//   out = sum_t softmax(scale q . k_t)_t v_t,   p - window < t <= p
//
// For sequences with more than kDecodeRows rows (new tokens times query heads of a
// KV head); fewer go to paged_decode.cu.
//
// One CTA per SM, persistent.  An item is one sequence's run of new tokens and one
// KV head: the rows are the tokens' query heads of that KV head, 128 a tensor-core
// tile, over the key tiles of 128 tokens that any row sees.  All items' key tiles
// form one line, cut into equal costs for the CTAs: a causal chunk's short and
// long rows balance, few rows over a long cache spread over all SMs, and an item
// that a cut divides is joined from f32 partials by merge_kernel (16 warps' blocks
// an item of 256 rows: one block alone took 13 to 30 us for 19 pieces).
//
// A CTA runs two softmax streams so that one's exponentials hide behind the other's
// products.  kPair (calls with more rows than a tile): two row tiles over the same
// keys, each key tile loaded once for 256 rows.  kOne (33 to 128 rows): one row
// tile, its key tiles taken in turn by the streams, which are joined at the item's
// end.
//
// Roles: warps 0-3 and 4-7 the streams' softmax, one row a thread (the row's
// logits sit in one tensor-memory lane, so no shuffles).  Warp 8 loads queries and
// keys by TMA, warp 11 values (pages land as they lie, 16 to 128 rows a box; one
// warp for both fell behind the products at pages of 16).  Warp 9, and in kPair
// warp 10 for the second stream, issue the products
//   S = Q K^T   shared x shared      O += P V   P from tensor memory
// S of one tile is overwritten in place by P, so two streams' S and O fill the 512
// columns.  int8: warp 8 loads keys and values as codes, warps 12-15 turn them into
// f16 or bf16.
//
// The reference m of a row's weights 2^(logit - m) follows its maximum loosely,
// from below: that spares the search for each tile's maximum, makes the rescaling of
// O rare, and leaves small weights the range of f16 (lift_of).
// P is rounded to the tensor core's operand type, bf16 for bf16 caches and f16 for f16
// and int8 ones: half a step of each weight, and in f16 at least 2^-31 of the row's
// largest (int8: 2^-30 of it times ScaleUnit's unit).  Sums and statistics in f32 do not
// add to that.
//
// What bounds it.  128 channels in f16: the power limit; 2048 tokens over 32,768
// take 755 to 805 us back to back, by the GPU = 1.32 to 1.41 PFLOP/s (0.78 to 0.83 of
// what a plain matrix product sustains).  64 channels: the two softmax warps a
// scheduler has, not its products: 2 x 4001 tokens 94 us = 0.70 PFLOP/s.  int8:
// the codes' way through shared memory beside the softmax: 250 tokens over 130,250
// 544 us = 0.98 PFLOP/s.  Few key tiles an SM: the set-up (2.5 us), an item's first
// loads and its last rows: 24 ragged sequences in a window 122 us = 0.81 PFLOP/s.
// The roles' code together is near the instruction cache's size, so each stays
// rolled and in one place: unrolling a role has cost others more than it gained.
#include <type_traits>

#include "paged_attn_dev.cuh"

namespace kvd {
namespace {

// A tile of rows has kTile of them too.
constexpr int kProducer = 8, kIssuer = 9;  // warps; the issuer of stream 1: 10
constexpr int kValueProducer = 11;         // f16 and bf16 caches: value tiles
enum Mode { kPair, kOne };  // how a call's rows lie on the tiles (see above)
// Registers a thread: 168 at launch (64,512 for 384 threads), or 128 (65,536 for
// 512), moved to the softmax warps, which hold a row's 128 logits:
// 256 * 208 + 128 * 88 = 64,512, or 256 * 184 + 256 * 72 = 65,536.
constexpr int threads_of(bool i8) { return i8 ? 512 : 384; }
constexpr int softmax_regs(bool i8) { return i8 ? 184 : 208; }
constexpr int other_regs(bool i8) { return i8 ? 72 : 88; }
constexpr int kTeam = 12, kTeamWarps = 4;  // warps that turn int8 codes
// A row's weights are 2^(logit - m).  m is set `lift` places below the row's maximum:
// f16 holds numbers from 2^-24 (with all their bits from 2^-14) to 2^16, and a row
// whose largest weight is an early key's (a sink's, say) has millions of small ones.  A
// tile whose weights add up to more than kRaise (twice 128 weights of 2^lift) raises m
// for the next one, and one above kRedo is computed again.  What has to fit is then
// kRedo, and for int8 kRedo times a value scale below 2 (ScaleUnit).  Restated on the
// host for one key with 0.99 of 131,072 keys' weight, what the others add is off by
// 2.7 % with lift 0, 0.007 % with 5 and 0.003 % with 6.
constexpr float lift_of(bool i8) { return i8 ? 5.0f : 6.0f; }

struct Dev : AttnArgs {
    int q_tokens;       // tokens of a row tile: 128 / G (kPair), or max_new
    float *acc;         // partial sums [2 * CTAs][rows / 32][D / 4][32][4]
    float2 *ml;         // their maxima and sums [2 * CTAs][rows]
    int4 *merge;        // [CTAs][2]: what merge_kernel joins
    int ws_rows;        // rows of a partial: 256 (PAIR) or fewer, a multiple of 32
};

// ---------------------------------------------------------------- items ---
struct Item {
    int i0, cnt;   // tokens of the sequence's new ones
    int lo, hi;    // keys [lo, hi) that any of them sees
    int j0, tiles; // key tiles: one at least, so that rows that see nothing are written
};

__device__ __forceinline__ Item item_of(const Dev &a, const Seq &s, int tile, int width) {
    Item it;
    it.i0 = tile * width;
    it.cnt = min(width, s.n - it.i0);
    const int p0 = s.first + it.i0;
    it.hi = max(p0 + it.cnt, 0);
    it.lo = a.window > 0 ? min(max(p0 - a.window + 1, 0), it.hi) : 0;
    it.j0 = it.lo / kTile;
    it.tiles = max((it.hi + kTile - 1) / kTile - it.j0, 1);
    return it;
}

// What an item takes beside its key tiles (its queries' way in, the first products
// and its rows' way out), in key tiles: the line is cut by tiles and these together,
// an item's first kItemCost units standing for it.  Cut by tiles alone the CTAs with
// many short items were the last by far (SMs busy 0.76 of the time); at 0, 1, 2, 3, 4
// and 6 units 2 x 4001 tokens at 64 channels took 109, 97, 93, 94, 95.5 and 97 us, 24
// ragged sequences 131, 123, 121, 121, 121 and 124.
constexpr int kItemCost = 3;

// A CTA's walk along the line of items, the same in every role.
struct Walk {
    int b, head, tile;
    int off;    // units of the item that lie before
    long left;  // units
    int k;  // segments taken
    Seq s;
};
struct Segment {
    Item it;
    int b, s0, first_pos, head;
    int j0, j1;        // key tiles
    bool starts, ends; // whether it holds its item's first and last tile
    int k;
};

__device__ __forceinline__ bool next_segment(const Dev &a, int width, Walk &w, Segment &g) {
    if (w.left <= 0) return false;
    g.it = item_of(a, w.s, w.tile, width);
    const int units = g.it.tiles + kItemCost;
    const int take = static_cast<int>(min(static_cast<long>(units - w.off), w.left));
    // the item's tiles are another CTA's: it begins with its first tile
    if (w.off + take <= kItemCost) return false;
    g.b = w.b;
    g.s0 = w.s.s0;
    g.first_pos = w.s.first;
    g.head = w.head;
    g.j0 = g.it.j0 + max(w.off - kItemCost, 0);
    g.j1 = g.it.j0 + w.off + take - kItemCost;
    g.starts = w.off <= kItemCost;
    g.ends = w.off + take == units;
    g.k = w.k++;
    w.left -= take;
    w.off = 0;
    if (w.left > 0) {
        if ((w.tile + 1) * width < w.s.n) {
            ++w.tile;
        } else {
            w.tile = 0;
            if (++w.head == a.c.n_kv_heads) {
                w.head = 0;
                do {
                    ++w.b;
                    if (w.b >= a.c.batch) {  // the line has no more items
                        w.left = 0;
                        break;
                    }
                    w.s = seq_of(a, w.b, false);
                } while (w.s.n == 0);
            }
        }
    }
    return true;
}

constexpr int kFewSeqs = 48;  // sequences whose row tiles are counted a warp each

// 32 bytes; wide: on a 32-byte boundary, in one store (the lanes' rows lie apart, so
// a store takes the L1 as many cycles as it has lanes, whatever it brings).
__device__ __forceinline__ void store32(void *p, const uint32_t (&w)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
                     "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        static_cast<uint4 *>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4 *>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// ------------------------------------------------------------ the kernel ---
template <int D, Mode MODE, bool I8>
struct Shape {
    static constexpr bool PAIR = MODE == kPair;
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kQHalf = kTile * 128;  // 64 channels of a row tile
    static constexpr int kQTile = kQHalf * (D / 64);
    static constexpr int kQBytes = (PAIR ? 2 : 1) * kQTile;
    static constexpr int kJoinBytes = PAIR ? 0 : kTile * 64 * 4;  // 64 channels of a stream's O
    static constexpr int kStages = I8 ? (D == 128 ? 3 : 6) : (D == 128 ? 5 : 8);
    // int8: tiles as loaded (codes, then the rows' key and value scales with keys),
    // and the scales the softmax takes, for more key tiles than the ring lets the
    // loads run ahead of it
    static constexpr int kRaw = !I8 ? 0 : D == 128 ? 3 : 6;
    static constexpr int kRawBytes = kTile * (D + 8);
    static constexpr int kScales = D == 128 ? 4 : 8;
    static constexpr int kScaleBytes = I8 ? kScales * 2 * kTile * 4 : 0;
    static constexpr int kAhead = PAIR ? 1 : 2;  // key tiles whose S is issued ahead of PV
    // +1024: the tiles start on a 1024-byte boundary
    static constexpr int kSmem = 1024 + kQBytes + kJoinBytes + kStages * kTileBytes +
                                 kRaw * kRawBytes + kScaleBytes;
};

struct Bars {
    uint64_t q_full[2], q_empty, kv_full[8], kv_empty[8], s_full[2], p_full[2], o_full[2], turn[2], done,
        join_full, join_empty, raw_full[8], raw_empty[8];
};

template <bool BF16, int D, Mode MODE, bool I8>
__global__ void __launch_bounds__(threads_of(I8), 1)
attn_kernel(const __grid_constant__ Dev a, const __grid_constant__ CUtensorMap q_map,
            const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
    using Sh = Shape<D, MODE, I8>;
    constexpr bool PAIR = MODE == kPair;
    // int8: weights and value codes are f16 whatever the queries are (three more
    // bits, and the codes take fewer instructions)
    constexpr bool kPBf16 = BF16 && !I8;
    constexpr float kLift = lift_of(I8);
    constexpr float kRaise = I8 ? 8192.0f : 16384.0f, kRedo = 2.0f * kRaise;  // 2^(lift + 8)
    constexpr int kThreads = threads_of(I8);
    constexpr int kHalves = D / 64;
    constexpr int kHalfBytes = kTile * 128;
    constexpr int kStages = Sh::kStages;
    constexpr int kAhead = Sh::kAhead;

    extern __shared__ uint8_t raw_smem[];
    __shared__ Bars bar;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    __shared__ uint32_t dead_groups[8];  // per key tile: its 16-key groups on bad pages
    __shared__ float2 join_ml[kTile];
    __shared__ int value_exp[8];            // int8: per key tile, see Scales
    __shared__ __align__(16) float ones[I8 ? kTile : 1];
    __shared__ long scan_total[kThreads / 32];
    __shared__ long seq_tiles[kFewSeqs];
    __shared__ long found_rest;
    __shared__ int found_seq;
    __shared__ Walk start;
    __shared__ uint4 loads[2];  // the loading warps' last: places and parities, of queries too

    uint8_t *smem = raw_smem + ((1024 - (smem_addr(raw_smem) & 1023)) & 1023);
    uint8_t *q_smem = smem;
    float *join = reinterpret_cast<float *>(smem + Sh::kQBytes);
    uint8_t *ring = smem + Sh::kQBytes + Sh::kJoinBytes;
    uint8_t *raw = ring + kStages * Sh::kTileBytes;
    // Scales: [kScales][2][128], a key tile's key scales times the softmax scale, and
    // its value scales times 2^-value_exp
    float *scales = reinterpret_cast<float *>(raw + Sh::kRaw * Sh::kRawBytes);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int width = PAIR ? 2 * a.q_tokens : a.q_tokens;  // tokens of an item

    if (warp == kIssuer) tmem_alloc(&tmem_slot, 512);
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.q_full[i], 1);
            mbar_init(&bar.s_full[i], 1);
            mbar_init(&bar.p_full[i], 4);
            mbar_init(&bar.o_full[i], 1);
            mbar_init(&bar.turn[i], 1);
        }
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bar.kv_full[i], I8 ? kTeamWarps : 2);
            mbar_init(&bar.kv_empty[i], PAIR ? 2 : 1);  // the streams that use a tile
        }
        for (int i = 0; i < Sh::kRaw; ++i) {
            mbar_init(&bar.raw_full[i], 1);
            mbar_init(&bar.raw_empty[i], kTeamWarps);
        }
        mbar_init(&bar.q_empty, PAIR ? 2 : 1);  // the warps that issue products
        mbar_init(&bar.done, PAIR ? 2 : 1);
        mbar_init(&bar.join_full, 4);
        mbar_init(&bar.join_empty, 4);
        fence_barrier_init();
        abort_flag = 0;
        start.left = 0;
    }
    if (I8 && tid < kTile) ones[tid] = 1.0f;
    pdl_wait();
    pdl_launch_dependents();

    // ---- this CTA's piece of the line of items
    // of one head of a sequence: a warp's lanes take a row tile each
    auto units_of = [&](const Seq &s) -> long {
        long n = 0;
#pragma unroll 1
        for (int t = lane; t * width < s.n; t += 32) n += item_of(a, s, t, width).tiles + kItemCost;
#pragma unroll
        for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
        return n;
    };
    // A lane's sequence: by itself up to kAlone row tiles, with the warp above.  49
    // sequences, one of them with 1000 row tiles in a window of 128: 84 us by itself, 60
    // with the warp; 49 with 2 or 4 each: 16 and 22 us by themselves, 23 and 29 with it.
    constexpr int kAlone = 16;
    auto cost_of = [&](int b, bool report) -> long {
        Seq s = {};
        if (b < a.c.batch) s = seq_of(a, b, report);
        const bool many = s.n > kAlone * width;
        long n = 0;
#pragma unroll 1
        for (int t = 0; !many && t * width < s.n; ++t)
            n += item_of(a, s, t, width).tiles + kItemCost;
        uint32_t more = __ballot_sync(0xffffffffu, many);
#pragma unroll 1
        for (; more; more &= more - 1) {
            const int l = __ffs(more) - 1;
            const long u = units_of(seq_of(a, b - lane + l, false));
            if (lane == l) n = u;
        }
        return n * a.c.n_kv_heads;
    };
    auto scan = [&](long cost, long &before) -> long {  // exclusive prefix, and the sum
        long v = cost;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        if (lane == 31) scan_total[warp] = v;
        __syncthreads();
        long sum = 0;
        before = v - cost;
        for (int i = 0; i < kThreads / 32; ++i) {
            if (i < warp) before += scan_total[i];
            sum += scan_total[i];
        }
        __syncthreads();
        return sum;
    };
    long before = 0;
    long cost;
    if (a.c.batch <= kFewSeqs) {
        // few sequences may be long: a warp counts one's tiles, a lane a row tile
#pragma unroll 1
        for (int b = warp; b < a.c.batch; b += kThreads / 32) {
            const long n = units_of(seq_of(a, b, blockIdx.x == 0));
            if (lane == 0) seq_tiles[b] = n;
        }
        __syncthreads();
        cost = tid < a.c.batch ? seq_tiles[tid] * a.c.n_kv_heads : 0;
    } else {
        cost = cost_of(tid, blockIdx.x == 0);
    }
    long total = scan(cost, before);
    const bool one_pass = a.c.batch <= kThreads;
#pragma unroll 1
    for (int b0 = kThreads; b0 < a.c.batch; b0 += kThreads) {
        long skip;
        total += scan(cost_of(b0 + tid, blockIdx.x == 0), skip);
    }
    const long per = max((total + gridDim.x - 1) / gridDim.x, static_cast<long>(a.min_tiles));
    const long ctas = max(min(static_cast<long>(gridDim.x), (total + per - 1) / per), 1l);
    const long share = total / ctas, spare = total % ctas;
    auto cut = [&](long c) { return c * share + min(c, spare); };  // where CTA c begins
    const long x0 = blockIdx.x < ctas ? cut(blockIdx.x) : total;
    const long x1 = blockIdx.x < ctas ? cut(blockIdx.x + 1) : total;
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
                found_seq = b0 + tid;
                found_rest = x0 - before;
                seq_tiles[0] = cost / a.c.n_kv_heads;  // of one head
            }
        }
        __syncthreads();
        if (warp == 0) {  // the row tile, 32 at a time
            Walk w;
            w.b = found_seq;
            w.s = seq_of(a, w.b, false);
            const long per_head = seq_tiles[0];
            w.head = static_cast<int>(found_rest / per_head);
            long r = found_rest - w.head * per_head;
#pragma unroll 1
            for (int t0 = 0;; t0 += 32) {
                const int t = t0 + lane;
                const int n = t * width < w.s.n ? item_of(a, w.s, t, width).tiles + kItemCost : 0;
                int upto = n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int u = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += u;
                }
                const uint32_t in = __ballot_sync(0xffffffffu, r < upto);
                if (in || t0 * width >= w.s.n) {
                    const int l = in ? __ffs(in) - 1 : 0;
                    w.tile = t0 + l;
                    w.off = static_cast<int>(r) - __shfl_sync(0xffffffffu, upto - n, l);
                    break;
                }
                r -= __shfl_sync(0xffffffffu, upto, 31);
            }
            w.left = x1 - x0;
            w.k = 0;
            if (lane == 0) start = w;
        }
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = tmem_slot;
    Walk w = start;
    Segment g;
    volatile int *abort = &abort_flag;
    auto fail = [&] {
        *abort = 1;
        report_status(a.c.dev_status, KVD_ERR_TIMEOUT);
    };

    // rows and key tiles of stream t in a segment
    struct Part {
        int cnt, p0, j0, j1;  // tokens, first position, key tiles (PAIR: its own; else the segment's)
    };
    auto part_of = [&](const Segment &g, int t) -> Part {
        Part p;
        const int i = g.it.i0 + (PAIR ? t * a.q_tokens : 0);
        p.cnt = min(a.q_tokens, g.it.i0 + g.it.cnt - i);
        p.p0 = g.first_pos + i;
        p.j0 = g.j0;
        p.j1 = g.j1;
        if constexpr (PAIR) {
            if (p.cnt <= 0) {
                p.cnt = 0;
                p.j1 = p.j0;
                return p;
            }
            const int hi = max(p.p0 + p.cnt, 0);
            const int lo = a.window > 0 ? min(max(p.p0 - a.window + 1, 0), hi) : 0;
            p.j0 = max(p.j0, lo / kTile);
            p.j1 = min(p.j1, (hi + kTile - 1) / kTile);
            if (p.j1 < p.j0) p.j1 = p.j0;
        }
        return p;
    };
    // the key tiles a segment loads: those some stream takes
    auto span_of = [&](const Segment &g, int &j0, int &j1) {
        j0 = g.j0;
        j1 = g.j1;
        if constexpr (PAIR) {
            const Part p0 = part_of(g, 0), p1 = part_of(g, 1);
            const bool e0 = p0.j0 == p0.j1, e1 = p1.j0 == p1.j1;
            if (e0 && e1) {
                j1 = j0;
            } else {
                j0 = e0 ? p1.j0 : e1 ? p0.j0 : min(p0.j0, p1.j0);
                j1 = e0 ? p1.j1 : e1 ? p0.j1 : max(p0.j1, p1.j1);
            }
        }
    };

    if (warp >= kProducer) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(other_regs(I8)));
        if (warp == kProducer || (!I8 && warp == kValueProducer)) {
        // ------------------------------------------------------- loads ---
        const bool first_warp = warp == kProducer;  // keys and all else
        const uint64_t policy = PAIR ? l2_policy_evict_last() : l2_policy_evict_first();
        const int boxes = kTile / a.box;
        const int ahead_tiles = 32 / boxes;  // whose rows one read of the page table gives
        const int ps = a.c.page_size;
        constexpr uint32_t kRawPlaces = I8 ? Sh::kRaw : 1;
        uint32_t st = 0, keys = 0;  // the next place (int8: of the raw ring), key tiles loaded
        uint32_t it = 0;            // int8: tiles loaded
        // Bits of the ring's places: whether one was used before, and the parity of
        // its next release.  Releases come in the order of the tiles, so a warp that
        // waits for every second one never falls a whole turn behind.
        uint32_t used = 0, phase = 0;
        uint32_t filled = 0, fills = 0;  // places whose full barrier was used; its next parity
        uint32_t q_filled = 0, q_fills = 0;  // and q_full's
        uint32_t q_phase = 0;
        bool ok = true;
        int4 rec0 = make_int4(0, 0, 0, 0), rec1 = make_int4(0, 0, 0, 0);
#pragma unroll 1
        while (ok && next_segment(a, width, w, g)) {
            int j0, j1;
            span_of(g, j0, j1);
            if (first_warp && g.k > 0) {
                ok = wait_for(&bar.q_empty, q_phase, abort);
                q_phase ^= 1;
                if (!ok) break;
            }
            if (first_warp && lane == 0 && j1 > j0) {
                const int rows = a.q_tokens * a.G;
#pragma unroll 1
                for (int t = 0; t < (PAIR ? 2 : 1); ++t) {
                    const Part p = part_of(g, t);
                    if (p.j0 == p.j1) continue;
                    q_filled |= 1u << t;
                    q_fills ^= 1u << t;
                    mbar_arrive_expect_tx(&bar.q_full[t], rows * 128 * kHalves);
#pragma unroll 1
                    for (int h = 0; h < kHalves; ++h)
                        tma_load_4d(q_smem + t * Sh::kQTile + h * Sh::kQHalf, &q_map, h * 64, 0,
                                    g.head, g.s0 + g.it.i0 + (PAIR ? t * a.q_tokens : 0),
                                    &bar.q_full[t]);
                }
            }
            // The cache rows of the boxes of tiles j, j + 1, .., a lane a box: dead_row
            // where none is needed, -1 on a bad page.
            auto rows_of = [&](int j) -> int {
                const int t0 = (j + lane / boxes) * kTile + lane % boxes * a.box;
                if (t0 >= j1 * kTile || t0 >= g.it.hi || t0 + a.box <= g.it.lo)
                    return a.dead_row;
                const int col = t0 / ps;
                const int page = checked_page(a.c, g.b, col);
                return page < 0 ? -1 : (page * a.c.n_kv_heads + g.head) * ps + (t0 - col * ps);
            };
            // int8: the tile's codes as they lie, and with keys both rows' scales
            auto load_raw = [&](int row, const CUtensorMap *map, bool keys_too) -> bool {
                if (it >= kRawPlaces) {
                    if (!wait_for(&bar.raw_empty[st], phase >> st & 1, abort)) return false;
                    phase ^= 1u << st;
                }
                const bool live = keys_too && lane < boxes && row != a.dead_row;
                const int n = __popc(__ballot_sync(0xffffffffu, live));
                filled |= 1u << st;
                fills ^= 1u << st;
                if (lane == 0)
                    mbar_arrive_expect_tx(&bar.raw_full[st], kTile * D + n * a.box * 8);
                __syncwarp();
                uint8_t *dst = raw + st * Sh::kRawBytes;
                if (lane < boxes)
                    tma_load_2d(dst + lane * a.box * D, map, 0, row, &bar.raw_full[st], policy);
                if (live) {
                    float *sc = reinterpret_cast<float *>(dst + kTile * D) + lane * a.box;
                    tma_load_1d(sc, static_cast<const float *>(a.c.k_scale) + row, a.box * 4,
                                &bar.raw_full[st], policy);
                    tma_load_1d(sc + kTile, static_cast<const float *>(a.c.v_scale) + row,
                                a.box * 4, &bar.raw_full[st], policy);
                }
                ++it;
                st = st + 1 == kRawPlaces ? 0 : st + 1;
                return true;
            };
            // The tiles in the order of the products: kAhead key tiles, then value
            // and key tiles in turn.  Rows are read ahead of their use.
            int kj = j0, vj = j0;
            int rows_k = 0, rows_v = 0, rows_next = rows_of(j0);
            uint64_t *full = nullptr;
#pragma unroll 1
            while (ok && vj < j1) {
                const bool is_k = kj < min(j1, vj + kAhead);
                const bool pre = vj == j0;  // a key tile before any value tile
                const int in = ((is_k ? kj : vj) - j0) % ahead_tiles;
                if (in == 0) {
                    if (is_k) {
                        rows_k = rows_next;
                        rows_next = rows_of(kj + ahead_tiles);
                    } else {
                        rows_v = rows_k;
                    }
                }
                int row = __shfl_sync(0xffffffffu, is_k ? rows_k : rows_v,
                                      in * boxes + lane % boxes);
                const bool bad = row < 0;
                if (bad) row = a.dead_row;
                if (is_k) {
                    const int n = a.box / 16;
                    const uint32_t groups = __reduce_or_sync(
                        0xffffffffu, bad ? ((1u << n) - 1) << (lane % boxes * n) : 0u);
                    if (lane == 0 && first_warp) dead_groups[keys & 7] = groups;
                    ++keys;
                    ++kj;
                } else {
                    ++vj;
                }
                const CUtensorMap *map = is_k ? &k_map : &v_map;
                if constexpr (I8) {
                    ok = load_raw(row, map, is_k);
                } else {
                    // The next place of the ring.  A value tile, and the key tile that
                    // follows it in the same step of the products, complete on the value
                    // tile's barrier; the first key tiles on their own.  A barrier counts
                    // two arrivals: of both tiles' warps, or of one warp twice.
                    const bool again = used >> st & 1;
                    const uint32_t parity = phase >> st & 1;
                    if (again) phase ^= 1u << st;
                    used |= 1u << st;
                    if (!is_k || pre) {
                        full = &bar.kv_full[st];
                        filled |= 1u << st;
                        fills ^= 1u << st;
                    }
                    if (is_k == first_warp) {
                        if (again && !(ok = wait_for(&bar.kv_empty[st], parity, abort))) {
                            fills ^= 1u << (full - bar.kv_full);  // not loaded
                            break;
                        }
                        if (lane == 0) {
                            mbar_arrive_expect_tx(full, Sh::kTileBytes);
                            if (is_k ? pre : kj == j1) mbar_arrive(full);
                        }
                        __syncwarp();
                        if (lane < boxes)
#pragma unroll
                            for (int h = 0; h < kHalves; ++h)
                                tma_load_2d(ring + st * Sh::kTileBytes + h * kHalfBytes +
                                                lane * a.box * 128,
                                            map, h * 64, row, full, policy);
                    }
                    st = st + 1 == kStages ? 0 : st + 1;
                }
            }
            if (g.starts && !g.ends) {
                // the item goes on in the next CTAs: leave word for merge_kernel
                const long rest = g.it.j0 + g.it.tiles - g.j1;  // tiles, and units
                int pieces = 1;
                while (cut(blockIdx.x + pieces + 1) - x1 < rest) ++pieces;
                rec0 = make_int4(pieces + 1, g.k == 0 ? 0 : 1, g.s0 + g.it.i0, g.it.cnt);
                rec1 = make_int4(g.head, 0, 0, 0);
            }
        }
        if (!ok) fail();
        if (lane == 0 && first_warp) {
            a.merge[2 * blockIdx.x] = rec0;
            a.merge[2 * blockIdx.x + 1] = rec1;
        }
        if (lane == 0) loads[first_warp] = make_uint4(filled, fills, q_filled, q_fills);
        } else if (warp == kIssuer || (PAIR && warp == kIssuer + 1)) {
            // ------------------------------------------------ products ---
            // An issued product waits until the tensor pipe has room, so a warp that
            // issues both streams' leaves the pipe idle through its own waits.  In
            // kPair, where the products are the bound, each stream has its warp, one
            // waiting behind the other's products; they take turns, which keeps one
            // stream's softmax beside the other's products.  Otherwise one warp
            // serves the streams' key tiles in turn.
            constexpr uint32_t kIdS = mma_idesc(BF16, kTile, kTile, false);
            constexpr uint32_t kIdO = mma_idesc(kPBf16, kTile, D, true);
            const int who = warp - kIssuer;  // kPair: the stream
            const uint32_t ring_addr = smem_addr(ring);
            const uint32_t q =
                warp_uniform(desc_low(smem_addr(q_smem + (PAIR ? who * Sh::kQTile : 0)), 16));
            uint32_t st = 0;          // place of the ring
            uint32_t full_phase = 0;  // bits of its places
            uint32_t q_phase = 0, p_phase = 0 /* bits: streams */, turn_phase = who ^ 1;
            bool ok = true;
            auto wait_tile = [&]() -> bool {  // what this place's barrier announces is there
                const bool r = wait_for(&bar.kv_full[st], full_phase >> st & 1, abort);
                full_phase ^= 1u << st;
                return r;
            };
            auto next_place = [&] { st = st + 1 == kStages ? 0 : st + 1; };
#pragma unroll 1
            while (ok && next_segment(a, width, w, g)) {
                int j0, j1;
                span_of(g, j0, j1);
                const Part part = part_of(g, who);
                // the warp's key tiles
                const int mine = PAIR ? part.j0 : j0, end = part.j1;
                auto takes = [&](int j) { return j >= mine && j < end; };
                constexpr int kStep = PAIR ? 1 : 2;  // to a stream's next tile
                if (mine < end) {
                    ok = wait_for(&bar.q_full[who], q_phase, abort);
                    q_phase ^= 1;
                } else {
                    if (elect_one()) mma_commit(&bar.q_empty);  // not read at all
                    __syncwarp();
                }
                // Step j: O of key tile j, and S of the one kAhead tiles on.
#pragma unroll 1
                for (int j = j0 - kAhead; ok && j < j1; ++j) {
                    const int ahead = j + kAhead;
                    const bool has_o = j >= j0, has_s = ahead < j1;
                    if (!has_o && !has_s) continue;
                    const int t = PAIR ? who : (j - j0) & 1;
                    const uint32_t s_at = warp_uniform(tmem + t * 128);
                    const bool do_o = has_o && takes(j), do_s = has_s && takes(ahead);
                    const uint32_t v_st = st;
                    const uint32_t v =
                        warp_uniform(desc_low(ring_addr + st * Sh::kTileBytes, kHalfBytes));
                    if (has_o) {
                        // the value tile, and the key tile ahead at the next place
                        if (!(ok = wait_tile())) break;
                        // value rows that no token of the item sees may hold NaN: clear them
                        // (each stream's warp, before its own product)
                        const int from = max(g.it.lo - j * kTile, 0);
                        const int to = min(g.it.hi - j * kTile, kTile);
                        if (!I8 && do_o && (from > 0 || to < kTile)) {
                            uint8_t *vs = ring + v_st * Sh::kTileBytes;
                            const int n = (from + (kTile - max(to, 0))) * 8 * kHalves;
#pragma unroll 1
                            for (int i = lane; i < n; i += 32) {
                                const int c = i % 8, h = (i / 8) % kHalves;
                                int r = i / (8 * kHalves);
                                if (r >= from) r += max(to, 0) - from;
                                *reinterpret_cast<uint4 *>(vs + h * kHalfBytes + r * 128 + c * 16) =
                                    make_uint4(0, 0, 0, 0);
                            }
                            fence_proxy_async();
                            __syncwarp();
                        }
                        next_place();
                    }
                    const bool own_k = has_s && (I8 || !has_o);  // a barrier of its own
                    if (own_k && !(ok = wait_tile())) break;
                    const uint32_t k = warp_uniform(desc_low(ring_addr + st * Sh::kTileBytes, 16));
                    const uint32_t add = warp_uniform(j >= mine + kStep);
                    if (do_o) {
                        if (!(ok = wait_for(&bar.p_full[t], p_phase >> t & 1, abort))) break;
                        p_phase ^= 1u << t;
                        tmem_fence_after();
                    }
                    if (PAIR) {
                        if (!(ok = wait_for(&bar.turn[t], turn_phase, abort))) break;
                        turn_phase ^= 1;
                    }
                    if (elect_one()) {
                        if (do_o) {
#pragma unroll
                            for (int i = 0; i < kTile / 16; ++i)
                                mma_ts(s_at + 256, s_at + i * 8, smem_desc(v + i * (2048 / 16)),
                                       kIdO, i > 0 ? 1 : add);
                            if (j + kStep >= end) mma_commit(&bar.o_full[t]);
                        }
                        if (do_s) {
#pragma unroll
                            for (int i = 0; i < D / 16; ++i) {
                                const uint32_t in = (i % 4) * 32;
                                mma_ss(s_at, smem_desc(q + ((i / 4) * Sh::kQHalf + in) / 16),
                                       smem_desc(k + ((i / 4) * kHalfBytes + in) / 16), kIdS,
                                       i > 0);
                            }
                            mma_commit(&bar.s_full[t]);
                        }
                        if (PAIR) mbar_arrive(&bar.turn[t ^ 1]);
                        // the tiles are used up, and with the last S the queries
                        if (has_o) mma_commit(&bar.kv_empty[v_st]);
                        if (has_s) mma_commit(&bar.kv_empty[st]);
                        if (do_s && ahead + 1 == end) mma_commit(&bar.q_empty);
                    }
                    __syncwarp();
                    if (has_s) next_place();
                }
            }
            if (!ok) fail();
            // every product and every barrier arrival is done before the CTA goes
            if (elect_one()) mma_commit(&bar.done);
            __syncwarp();
            volatile int none = 0;
            if (!mbar_wait(&bar.done, 0, &none)) fail();
        }
        if (I8 && warp >= kTeam) {
            const int place = warp - kTeam;
            // --------------------------------------------- int8 to f16 or bf16 ---
            // Codes are whole numbers up to 127, exact in either type; the scales
            // go to the softmax, so the products lose nothing.
            constexpr int kTeamThreads = 32 * kTeamWarps;
            constexpr uint32_t kRaw = I8 ? Sh::kRaw : 1;
            constexpr int kUnits = D / 16;                  // 16-code steps a row
            constexpr int kWarpRows = 32 / kUnits;          // rows a warp's step takes
            constexpr int kSteps = kTile / (kWarpRows * kTeamWarps);
            // This lane's row and 16 codes of a step.  The 8 lanes of a load or a
            // store lie on two rows: at D = 128 on the one's first half and the
            // other's second, so that the codes come from all banks; and as the
            // swizzle turns even chunks of an odd row into odd ones, the chunks go
            // to all banks too.
            const int q8 = lane >> 3, k8 = lane & 7;
            const int my_row = place * kWarpRows +
                               (D == 128 ? 2 * (q8 >> 1) + (k8 >> 2) : lane >> 2);
            const int my_u = D == 128 ? (k8 & 3) + 4 * ((q8 & 1) ^ (k8 >> 2)) : lane & 3;
            const int src_at = my_row * D + 16 * my_u;
            const int dst_row = (my_u / 4) * kHalfBytes + my_row * 128;
            const int dst0 = dst_row + 16 * (((my_u % 4) * 2) ^ (my_row & 7));
            const int dst1 = dst_row + 16 * (((my_u % 4) * 2 + 1) ^ (my_row & 7));
            constexpr int kStepRows = kWarpRows * kTeamWarps;  // a multiple of 8
            static_assert(kStepRows % 8 == 0, "the swizzle of a lane's row stays");
            const int ct = place * 32 + lane;
            uint32_t n = 0, keys = 0;  // tiles and key tiles so far
            ScaleUnit unit = {};
            bool ok = true;
            // The scales of key tile j for the softmax.
            auto turn_scales = [&](const float *sc, int j, bool first) {
                const uint32_t bad = dead_groups[keys & 7];
                const bool edge = j * kTile < g.it.lo || (j + 1) * kTile > g.it.hi || bad;
                auto dead = [&](int at) {
                    const int tok = j * kTile + at;
                    return tok < g.it.lo || tok >= g.it.hi || (bad >> (at / 16) & 1);
                };
                // the exponent of the tile's largest value scale (infinities and NaN
                // count for nothing); each warp looks at all 128
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t v = __float_as_uint(sc[kTile + i * 32 + lane]);
                    if (v < 0x7f800000u && !(edge && dead(i * 32 + lane))) top = max(top, v);
                }
                top = __reduce_max_sync(0xffffffffu, top);
                unit.take(top, first, 1);  // scales below 2: weights up to kRedo fit f16
                const float inv = __int_as_float((127 - unit.exp) << 23);
                float *to = scales + keys % Sh::kScales * (2 * kTile);
#pragma unroll
                for (int at = ct; at < kTile; at += kTeamThreads) {
                    float ks = sc[at] * a.scale_log2, vs = sc[kTile + at] * inv;
                    if (edge && dead(at)) ks = vs = 0.0f;
                    to[at] = ks;
                    to[kTile + at] = vs;
                }
                if (ct == 0) value_exp[keys % Sh::kScales] = unit.exp;
            };
            // Tile n.
            auto turn = [&](bool is_k, int j, bool first) -> bool {
                const uint32_t st = n % kStages, rs = n % kRaw;
                if (!wait_for(&bar.raw_full[rs], (n / kRaw) & 1, abort)) return false;
                if (n >= kStages && !wait_for(&bar.kv_empty[st], (n / kStages - 1) & 1, abort))
                    return false;
                const uint8_t *src = raw + rs * Sh::kRawBytes;
                if (is_k) turn_scales(reinterpret_cast<const float *>(src + kTile * D), j, first);
                src += src_at;
                uint8_t *dst = ring + st * Sh::kTileBytes;
                // rolled: the roles' hot lines have to stay in the instruction cache
                // together (unrolled 8 times a tile took 1.4 times as long)
                auto codes = [&](auto bf16_tag) {
                    constexpr bool kBf16 = decltype(bf16_tag)::value;
#pragma unroll 4
                    for (int i = 0; i < kSteps; ++i) {
                        const uint4 w = *reinterpret_cast<const uint4 *>(src + i * (kStepRows * D));
                        uint4 lo, hi;
                        codes_to<kBf16>(w.x, lo.x, lo.y);
                        codes_to<kBf16>(w.y, lo.z, lo.w);
                        codes_to<kBf16>(w.z, hi.x, hi.y);
                        codes_to<kBf16>(w.w, hi.z, hi.w);
                        *reinterpret_cast<uint4 *>(dst + dst0 + i * (kStepRows * 128)) = lo;
                        *reinterpret_cast<uint4 *>(dst + dst1 + i * (kStepRows * 128)) = hi;
                    }
                };
                if (BF16 && is_k)
                    codes(std::true_type());
                else
                    codes(std::false_type());
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bar.kv_full[st]);
                    mbar_arrive(&bar.raw_empty[rs]);
                }
                return true;
            };
#pragma unroll 1
            while (ok && next_segment(a, width, w, g)) {
                int j0, j1;
                span_of(g, j0, j1);
                int kj = j0, vj = j0;
#pragma unroll 1
                while (ok && vj < j1) {  // the order of the loads
                    const bool is_k = kj < min(j1, vj + kAhead);
                    ok = turn(is_k, kj, kj == j0);
                    ++n;
                    keys += is_k;
                    ++(is_k ? kj : vj);
                }
            }
            if (!ok) fail();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(softmax_regs(I8)));
        // ------------------------------------------------------ softmax ---
        const int t = warp >> 2, row = tid & 127;
        const uint32_t lanes = tmem + ((warp & 3) << 21);  // this warp's 32 lanes
        const uint32_t s_addr = lanes + t * 128, o_addr = lanes + 256 + t * 128;
        uint32_t s_phase = 0, o_phase = 0, join_phase = 0, keys = 0;
        const int tok = row / a.G, head_at = (row - tok * a.G) * D;  // of this row
        bool ok = true;
#pragma unroll 1
        while (ok && next_segment(a, width, w, g)) {
            int j0, j1;
            span_of(g, j0, j1);
            const Part part = part_of(g, t);
            const int rows = part.cnt * a.G;
            const bool warp_live = (warp & 3) * 32 < rows;
            const int pos = part.p0 + tok;
            // keys [lo, hi) of this row
            const int hi = row < rows ? max(pos + 1, 0) : 0x7fffffff;
            const int lo = row < rows && a.window > 0 ? max(pos - a.window + 1, 0) : 0;
            // Rows that are none (another sequence's queries stand there, or what the memory
            // held): weights of 0 or NaN, and so no say in the votes
            float m = row < rows ? -INFINITY : INFINITY;
            float l = 0.0f, last = 0.0f;
            const int first = PAIR ? part.j0 : j0 + t;
            int exp_now = 0;  // int8: O is in units of 2^exp_now
#pragma unroll 1
            for (int j = first; j < part.j1; j += PAIR ? 1 : 2) {
                if (!(ok = wait_for(&bar.s_full[t], s_phase, abort))) break;
                s_phase ^= 1;
                if (warp_live) {
                    tmem_fence_after();
                    // int8 holds half the row's logits, and reads the others from
                    // tensor memory again where they are used (P overwrites the
                    // first half only): the scales take registers too
                    constexpr int kHeld = I8 ? 2 : 4;
                    float s[32 * kHeld];
#pragma unroll
                    for (int i = 0; i < kHeld; ++i) tmem_ld32(s_addr + 32 * i, s + 32 * i);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < kHeld; ++i) pin32(s + 32 * i);
                    const int rh = hi - j * kTile, rl = lo - j * kTile;
                    const uint32_t dead = dead_groups[(keys + (j - j0)) & 7];
                    const float *tile_sc = scales + (keys + (j - j0)) % Sh::kScales * (2 * kTile);
                    // in a tile that hides keys from a row the logits are scaled
                    // before they are hidden (0 * infinity is none)
                    const bool hides = __any_sync(0xffffffffu, rh < kTile || rl > 0) || dead;
                    const float *k_sc = I8 && hides ? ones : tile_sc;
                    auto hide = [&](float *v, int c0) {
                        auto below = [](int n) {  // n low bits
                            return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1;
                        };
                        uint32_t seen = below(rh - c0) & ~below(rl - c0);
                        if (dead >> (c0 / 16) & 1) seen &= 0xffff0000u;
                        if (dead >> (c0 / 16) & 2) seen &= 0x0000ffffu;
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            if (I8) v[c] *= tile_sc[c0 + c];
                            if (!(seen >> c & 1)) v[c] = -INFINITY;
                        }
                    };
                    if (hides)
#pragma unroll
                        for (int i = 0; i < kHeld; ++i) hide(s + 32 * i, 32 * i);
                    int new_exp = 0;
                    if constexpr (I8) {
                        new_exp = value_exp[(keys + (j - j0)) % Sh::kScales];
                        if (j == first) exp_now = new_exp;
                    }
                    // The exponentials take the scale of the tiles before, and the
                    // tile's own sum tells whether it still fits: one above kRaise
                    // raises the scale for the next tile, one above kRedo (or a row's
                    // first tile) finds the maximum and computes the tile again.
                    // In between no pass over the row looks for a maximum.
                    bool fix = __any_sync(0xffffffffu, m == -INFINITY || last > kRaise) ||
                               (I8 && new_exp != exp_now);
                    float2 sum[2];
#pragma unroll 1
                    for (;;) {
                        if (fix) {
                            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                            auto top_of = [&](const float *v, int c0, int n) {
#pragma unroll
                                for (int c = 0; c < n; c += 8)
#pragma unroll
                                    for (int i = 0; i < 4; ++i)
                                        mx[i] = I8 ? fmax3(mx[i], v[c + i] * k_sc[c0 + c + i],
                                                           v[c + 4 + i] * k_sc[c0 + c + 4 + i])
                                                   : fmax3(mx[i], v[c + i], v[c + 4 + i]);
                            };
                            top_of(s, 0, 32 * kHeld);
                            if constexpr (I8) {
#pragma unroll 1
                                for (int i = kHeld; i < 4; ++i) {
                                    float v[32];
                                    tmem_ld32(s_addr + 32 * i, v);
                                    tmem_wait_ld();
                                    pin32(v);
                                    if (hides) hide(v, 32 * i);
                                    top_of(v, 32 * i, 32);
                                }
                            }
                            const float top = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]) *
                                                  (I8 ? 1.0f : a.scale_log2) -
                                              kLift;
                            const float mn = fmaxf(
                                last > kRaise ? m + __log2f(last) - (kLift + 7.0f) : m, top);
                            const float f = m == -INFINITY || mn == -INFINITY
                                                ? 1.0f
                                                : exp2_approx(m - mn);
                            m = mn;
                            last = 0.0f;
                            l *= f;
                            if (j > first) {
                                // up by at most 2^60 (ScaleUnit), down to 0 where it matters
                                const float fo =
                                    I8 ? f * exp2_approx(static_cast<float>(exp_now - new_exp)) : f;
#pragma unroll 1
                                for (int i = 0; i < D / 16; ++i) {
                                    float o[16];
                                    tmem_ld16(o_addr + 16 * i, o);
                                    tmem_wait_ld();
                                    pin16(o);
#pragma unroll
                                    for (int c = 0; c < 16; ++c) o[c] *= fo;
                                    tmem_st16(o_addr + 16 * i, reinterpret_cast<uint32_t *>(o));
                                }
                            }
                        }
                        exp_now = new_exp;
                        const float base = m == -INFINITY ? 0.0f : m;
                        const float2 sc = make_float2(a.scale_log2, a.scale_log2);
                        const float2 off = make_float2(-base, -base);
                        sum[0] = sum[1] = make_float2(0.0f, 0.0f);
                        // the weights of 32 keys, and P
                        auto weights = [&](const float *v, int c0) {
                            uint32_t p[16];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                float4 kc[4], vc[4];  // int8: the scales of 16 keys
                                if constexpr (I8) {
#pragma unroll
                                    for (int c = 0; c < 4; ++c) {
                                        const int at = c0 + 16 * h + 4 * c;
                                        kc[c] = *reinterpret_cast<const float4 *>(k_sc + at);
                                        vc[c] =
                                            *reinterpret_cast<const float4 *>(tile_sc + kTile + at);
                                    }
                                }
#pragma unroll
                                for (int c = 0; c < 8; ++c) {
                                    const int at = 16 * h + 2 * c;
                                    const float4 k4 = kc[c / 2], v4 = vc[c / 2];
                                    float2 x = __ffma2_rn(
                                        make_float2(v[at], v[at + 1]),
                                        !I8          ? sc
                                        : c % 2 == 0 ? make_float2(k4.x, k4.y)
                                                     : make_float2(k4.z, k4.w),
                                        off);
                                    x.x = exp2_approx(x.x);
                                    x.y = exp2_approx(x.y);
                                    sum[c & 1] = __fadd2_rn(sum[c & 1], x);
                                    if (I8)
                                        x = __fmul2_rn(x, c % 2 == 0 ? make_float2(v4.x, v4.y)
                                                                     : make_float2(v4.z, v4.w));
                                    p[8 * h + c] = pack2<kPBf16>(x.x, x.y);
                                }
                            }
                            tmem_st16(s_addr + c0 / 2, p);
                        };
                        if constexpr (I8) {
                            float v[2][32];
                            tmem_ld32(s_addr + 64, v[0]);
                            weights(s, 0);
                            tmem_ld32(s_addr + 96, v[1]);
                            weights(s + 32, 32);
                            tmem_wait_ld();
                            pin32(v[0]);
                            pin32(v[1]);
                            if (hides) {
                                hide(v[0], 64);
                                hide(v[1], 96);
                            }
                            weights(v[0], 64);
                            weights(v[1], 96);
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i) weights(s + 32 * i, 32 * i);
                        }
                        sum[0] = __fadd2_rn(sum[0], sum[1]);
                        last = sum[0].x + sum[0].y;
                        // after a fix no weight passes 2^lift
                        if (fix || !__any_sync(0xffffffffu, last > kRedo)) break;
                        fix = true;
                        last = 0.0f;
                    }
                    l += last;
                    tmem_wait_st();
                    tmem_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.p_full[t]);
            }
            if (!ok) break;
            keys += j1 - j0;
            // ---- the segment's result
            const bool some = first < part.j1;
            if (some) {
                if (!(ok = wait_for(&bar.o_full[t], o_phase, abort))) break;
                o_phase ^= 1;
                tmem_fence_after();
            }
            const bool whole = g.starts && g.ends;
            const int prow = (PAIR ? t * 128 : 0) + row;
            const size_t slot = 2 * blockIdx.x + (g.k == 0 ? 0 : 1);
            // scale of this stream's O and of the joined one's
            const float unit = I8 ? __int_as_float((127 + exp_now) << 23) : 1.0f;
            float mine = unit, other = 0.0f;
            if constexpr (!PAIR) {
                if (t == 1) {
                    // the halves of the segment before have been read
                    if (!(ok = wait_for(&bar.join_empty, join_phase ^ 1, abort))) break;
                    join_ml[row] = make_float2(m, l);
                }
                if (t == 0) {
                    if (!(ok = wait_for(&bar.join_full, join_phase, abort))) break;
                    const float2 o = join_ml[row];
                    const float mn = fmaxf(m, o.x);
                    mine = m == -INFINITY ? 0.0f : exp2_approx(m - mn);
                    other = o.x == -INFINITY ? 0.0f : exp2_approx(o.x - mn);
                    l = l * mine + o.y * other;
                    mine *= unit;
                    m = mn;
                }
            }
            const bool live = row < rows;
            if (whole && (PAIR || t == 0)) {
                const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
                mine = some ? mine * inv : 0.0f;
                other *= inv;
                if (a.lse && live)
                    *lse_at(a, g.s0 + g.it.i0 + (PAIR ? t * a.q_tokens : 0) + tok, g.head,
                            row - tok * a.G) = lse_of(m, l);
            }
            if ((PAIR || t == 0) && live && !whole) a.ml[slot * a.ws_rows + prow] = make_float2(m, l);
            uint16_t *dst = a.out;
            if (live)
                dst += static_cast<int64_t>(g.s0 + g.it.i0 + (PAIR ? t * a.q_tokens : 0) + tok) *
                           a.out_stride +
                       static_cast<int64_t>(g.head) * a.G * D + head_at;
            float4 *part_dst = reinterpret_cast<float4 *>(a.acc) +
                               ((slot * (a.ws_rows / 32) + prow / 32) * (D / 4)) * 32 + lane;
            const bool wide = (reinterpret_cast<uintptr_t>(dst) & 31) == 0;
            // 16 channels at a time, in short code: it runs once a segment, from
            // beyond the instruction cache
#pragma unroll 1
            for (int i = 0; i < D / 16; ++i) {
                if (!PAIR && i > 0 && i % 4 == 0) {  // the join buffer holds 64
                    ok = t == 1 ? wait_for(&bar.join_empty, join_phase ^ 1, abort)
                                : wait_for(&bar.join_full, join_phase, abort);
                    if (!ok) break;
                }
                float o[16];
                if (some) {
                    tmem_ld16(o_addr + 16 * i, o);
                    tmem_wait_ld();
                    pin16(o);
                }
                float *at = join + i % 4 * 16 * kTile + row;
#pragma unroll
                for (int c = 0; c < 16; ++c)
                    o[c] = some && (PAIR || mine != 0.0f) ? o[c] * mine : 0.0f;
                if constexpr (!PAIR) {
                    if (t == 1) {
#pragma unroll
                        for (int c = 0; c < 16; ++c) at[c * kTile] = o[c];
                    } else {
                        float u[16];
#pragma unroll
                        for (int c = 0; c < 16; ++c) u[c] = at[c * kTile];
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            if (other != 0.0f) o[c] = fmaf(u[c], other, o[c]);
                    }
                }
                if (live && (PAIR || t == 0)) {
                    if (whole) {
                        uint32_t w[8];
#pragma unroll
                        for (int c = 0; c < 8; ++c) w[c] = pack2<BF16>(o[2 * c], o[2 * c + 1]);
                        store32(dst + 16 * i, w, wide);
                    } else {
#pragma unroll
                        for (int c = 0; c < 16; c += 4)
                            part_dst[(4 * i + c / 4) * 32] =
                                make_float4(o[c], o[c + 1], o[c + 2], o[c + 3]);
                    }
                }
                __syncwarp();
                if (!PAIR && i % 4 == 3) {
                    if (lane == 0) mbar_arrive(t == 1 ? &bar.join_full : &bar.join_empty);
                    join_phase ^= 1;
                }
            }
        }
        if (!ok) fail();
    }
    tmem_fence_before();
    __syncthreads();
    if (*abort && (warp == kProducer || (!I8 && warp == kValueProducer))) {
        // nothing may land in shared memory after the CTA has gone
        const uint4 of = loads[warp == kProducer];
        volatile int none = 0;
        uint64_t *full = I8 ? bar.raw_full : bar.kv_full;
        // a wait that runs out is for the other warp's part of a barrier; by then all
        // has had the time to land
        bool landed = true;
        for (uint32_t st = 0; landed && st < 8; ++st)
            if (of.x >> st & 1) landed = mbar_wait(&full[st], ~(of.y >> st) & 1, &none);
        for (uint32_t t = 0; landed && t < 2; ++t)
            if (of.z >> t & 1) landed = mbar_wait(&bar.q_full[t], ~(of.w >> t) & 1, &none);
    }
    if (warp == kIssuer) {
        tmem_fence_after();
        tmem_free(tmem, 512);
    }
}

// Joins the items that a cut between CTAs divided: CTA (c, y) serves the item
// whose first piece is CTA c's last segment and goes on in the CTAs after it.
//   out = sum_i 2^(m_i - m) acc_i / sum_i 2^(m_i - m) l_i
// A warp takes 32 rows and 8 channels at a time, a lane a row.
template <bool BF16, int D>
__global__ void __launch_bounds__(256) merge_kernel(const __grid_constant__ Dev a) {
    pdl_wait();
    pdl_launch_dependents();
    const int4 rec = a.merge[2 * blockIdx.x];
    if (rec.x == 0) return;
    const int head = a.merge[2 * blockIdx.x + 1].x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int blocks = a.ws_rows / 32;
    const size_t first = 2 * blockIdx.x + rec.y, next = 2 * blockIdx.x;
    for (int u = blockIdx.y * 8 + warp; u < blocks * (D / 8); u += gridDim.y * 8) {
        const int prow = u / (D / 8) * 32 + lane, c8 = u % (D / 8);
        const int r = prow % kTile;
        const int tok = prow / kTile * a.q_tokens + r / a.G;
        if (r >= a.q_tokens * a.G || tok >= rec.w) continue;
        float m = -INFINITY;
#pragma unroll 8
        for (int i = 0; i < rec.x; ++i)
            m = fmaxf(m, a.ml[(i == 0 ? first : next + 2 * i) * a.ws_rows + prow].x);
        float o[8] = {};
        float l = 0.0f;
#pragma unroll 4
        for (int i = 0; i < rec.x; ++i) {
            const size_t slot = i == 0 ? first : next + 2 * i;
            const float2 ml = a.ml[slot * a.ws_rows + prow];
            const float f = ml.x == -INFINITY ? 0.0f : exp2_approx(ml.x - m);
            const float4 *p = reinterpret_cast<const float4 *>(a.acc) +
                              ((slot * blocks + prow / 32) * (D / 4) + 2 * c8) * 32 + lane;
            const float4 u0 = p[0], u1 = p[32];
            const float u[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
            l = fmaf(f, ml.y, l);  // a sum that is NaN stays one where f is 0
            if (f != 0.0f) {
#pragma unroll
                for (int c = 0; c < 8; ++c) o[c] = fmaf(f, u[c], o[c]);
            }
        }
        const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
        if (a.lse && c8 == 0) *lse_at(a, rec.z + tok, head, r % a.G) = lse_of(m, l);
        *reinterpret_cast<uint4 *>(a.out + static_cast<int64_t>(rec.z + tok) * a.out_stride +
                                   static_cast<int64_t>(head * a.G + r % a.G) * D + 8 * c8) =
            make_uint4(pack2<BF16>(o[0] * inv, o[1] * inv), pack2<BF16>(o[2] * inv, o[3] * inv),
                       pack2<BF16>(o[4] * inv, o[5] * inv), pack2<BF16>(o[6] * inv, o[7] * inv));
    }
}

// ----------------------------------------------------------------- launch ---
struct WsPlan {
    int ctas, rows;
    bool pair;
    size_t merge, ml, acc, total;
};

WsPlan ws_plan(int G, int D, int max_new) {
    WsPlan w;
    w.ctas = device_sm_count();
    w.pair = max_new > kTile / G;
    w.rows = w.pair ? 2 * kTile : (max_new * G + 31) / 32 * 32;
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    w.merge = paged_counter_bytes();
    w.ml = w.merge + up(static_cast<size_t>(w.ctas) * 2 * sizeof(int4));
    w.acc = w.ml + up(static_cast<size_t>(w.ctas) * 2 * w.rows * sizeof(float2));
    w.total = w.acc + up(static_cast<size_t>(w.ctas) * 2 * w.rows * D * sizeof(float));
    return w;
}

template <bool BF16, int D, Mode MODE, bool I8>
cudaError_t launch_shape(const PagedAttnArgs &p, const WsPlan &w, void *ws, cudaStream_t st) {
    Dev a = {};
    a.q_tokens = MODE == kPair ? kTile / p.G : p.max_new;
    CUtensorMap q_map, k_map, v_map;
    constexpr CUtensorMapSwizzle kv_swizzle =
        I8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B;
    if (!fill_launch(p, a.q_tokens, kv_swizzle, kv_swizzle, a, q_map, k_map, v_map))
        return cudaErrorInvalidValue;
    a.min_tiles = kItemCost + 1;  // an item's first CTA takes a tile
    uint8_t *base = static_cast<uint8_t *>(ws);
    a.merge = reinterpret_cast<int4 *>(base + w.merge);
    a.ml = reinterpret_cast<float2 *>(base + w.ml);
    a.acc = reinterpret_cast<float *>(base + w.acc);
    a.ws_rows = w.rows;

    constexpr size_t smem = Shape<D, MODE, I8>::kSmem;
    constexpr int threads = threads_of(I8);
    auto *kernel = attn_kernel<BF16, D, MODE, I8>;
    cudaError_t e = prepare_kernel(reinterpret_cast<const void *>(kernel), threads, smem);
    if (e != cudaSuccess) return e;
    e = launch_ex(kernel, dim3(w.ctas), dim3(threads), smem, st, true, a, q_map, k_map,
                  v_map);
    if (e != cudaSuccess) return e;
    return launch_ex(merge_kernel<BF16, D>, dim3(w.ctas, MODE == kPair ? 16 : 4), dim3(256), 0, st, true, a);
}

template <bool BF16, int D, bool I8>
cudaError_t launch_mode(const PagedAttnArgs &p, const WsPlan &w, void *ws, cudaStream_t st) {
    if (w.pair) return launch_shape<BF16, D, kPair, I8>(p, w, ws, st);
    return launch_shape<BF16, D, kOne, I8>(p, w, ws, st);
}

template <bool BF16, bool I8>
cudaError_t launch_type(const PagedAttnArgs &p, void *ws, cudaStream_t st) {
    const WsPlan w = ws_plan(p.G, p.c.head_dim, p.max_new);
    return p.c.head_dim == 64 ? launch_mode<BF16, 64, I8>(p, w, ws, st)
                              : launch_mode<BF16, 128, I8>(p, w, ws, st);
}

}  // namespace

cudaError_t launch_paged_attn(const PagedAttnArgs &a, void *ws, cudaStream_t st) {
    if (a.c.dtype == KVD_INT8)
        return a.bf16 ? launch_type<true, true>(a, ws, st) : launch_type<false, true>(a, ws, st);
    return a.bf16 ? launch_type<true, false>(a, ws, st) : launch_type<false, false>(a, ws, st);
}

size_t paged_attn_ws(const kvd_paged_cache &c, int H, int max_new) {
    return ws_plan(H / c.n_kv_heads, c.head_dim, max_new).total;
}

}  // namespace kvd
