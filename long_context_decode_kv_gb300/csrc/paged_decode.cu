// paged_decode.cu -- attention over a paged cache for few rows: single tokens and
// short runs of new ones, whose query heads of one KV head number at most 32.
//
//   out = sum_t softmax(scale q . k_t)_t v_t,   p - window < t <= p
//
// Bound by the cache's bytes, so the keys take the tensor core's 128 lanes and the
// rows its narrow side: S^T = K Q^T and O^T = V^T P^T cost a quarter to an eighth
// of what row tiles would, and a thread holds one key's logits.  Its key and value
// scales (int8) are then two numbers of its own, its exponentials as many as there
// are rows, and the sums over keys stay apart until the end.
//
// One CTA per SM, persistent; the line of all items' (sequence, KV head) key tiles is
// cut into equal pieces; an item that a cut divides is joined by the last of its CTAs
// to arrive, from f32 partials.
//
// Roles: warps 0-3 softmax (thread = key); warps 4 and 5 load key and value tiles
// by TMA, a ring each; warps 6 and 7 issue the two products.  int8: warps 8-11
// turn key codes into f16 or bf16 whole numbers in tensor memory, where the
// product takes its first operand from, and warps 12-15 value codes in shared
// memory.  Keys that went through shared memory once more (64 KB of the tile's
// 200) would cost it more time than HBM takes for the tile.  The scales are read
// by the warps that turn the keys: as copies of a page's 16 to 128 numbers they
// would keep the loading warp longer than the codes do.
//
// The weights' reference m follows a row's maximum loosely, from kLift places below it
// (f16's range, see paged_attn.cu): a weight that passes kRedo (rarely any) has the
// four warps find the maximum and compute the tile again, as the first tile of an item
// does, and each one until all rows have seen a key (a window or a bad page may hide
// the first tiles from some).
//
// Measured: 8 sequences of 131,072 tokens, 32 heads over 8: 364 us int8 (6.1 TB/s,
// 0.89 of what a copy reaches; 460 with bf16 queries, whose key codes take 8
// instructions for four where f16's take 5), 613 us f16 (7.0 TB/s).  A decode step on
// 4 int8 sequences of 32,000, with its append, takes 68 us (0.58): a CTA's 20 tiles
// then stand beside the set-up, the first bytes and the join.  One token over 512: 8.3
// us, of which a launch and its host call are 5.
#include "paged_attn_dev.cuh"

namespace kvd {
namespace {

constexpr int kMaxCtas = 256;     // one an SM
constexpr float kLift = 6.0f;     // a new reference: so far below the row's maximum

// Barriers of the 128 softmax threads; the second tells whether any said yes.
__device__ __forceinline__ void meet_128() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool any_of_128(bool mine) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
        "bar.red.or.pred p, 1, 128, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(mine))
        : "memory");
    return r != 0;
}

struct DecodeArgs : AttnArgs {
    uint32_t *arrived;  // [CTAs], zero between calls: pieces of the item that CTA c's last
                        // segment begins
    float2 *ml;         // [2 * CTAs][NR] references and sums of partials
    float *acc;         // [2 * CTAs][NR][D]
};

// A CTA's walk along the line of items' key tiles.
struct Place {
    int b, head, off;
    int left;  // tiles
    Seq s;
};
struct Run {  // tiles [j0, j1) of an item, from its tile `off` on
    int j0, j1, lo, hi, tiles, off;
    int b, head;
    Seq s;
};

__device__ __forceinline__ Run run_of(const AttnArgs &a, const Seq &s) {
    Run r;
    r.hi = max(s.first + s.n, 0);
    r.lo = a.window > 0 ? min(max(s.first - a.window + 1, 0), r.hi) : 0;
    r.j0 = r.lo / kTile;
    r.tiles = max((r.hi + kTile - 1) / kTile - r.j0, 1);
    return r;
}

// The next run of the walk, or false at its end.
__device__ __forceinline__ bool next_run(const AttnArgs &a, Place &p, Run &r) {
    if (p.left <= 0) return false;
    r = run_of(a, p.s);
    const int take = min(r.tiles - p.off, p.left);
    r.off = p.off;
    r.j0 += p.off;
    r.j1 = r.j0 + take;
    r.b = p.b;
    r.head = p.head;
    r.s = p.s;
    p.left -= take;
    p.off = 0;
    if (p.left > 0 && ++p.head == a.c.n_kv_heads) {
        p.head = 0;
#pragma unroll 1
        do {
            if (++p.b >= a.c.batch) {
                p.left = 0;
                break;
            }
            p.s = seq_of(a, p.b, false);
        } while (p.s.n == 0);
    }
    return true;
}

template <int D, int NR, bool I8>
struct DecodeShape {
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kQHalf = NR * 128;            // 64 channels of the rows
    static constexpr int kQBytes = kQHalf * (D / 64);
    static constexpr int kPBytes = NR * 256;           // weights of a tile
    // keys: as the product takes them, or (int8) codes
    static constexpr int kKeyBytes = I8 ? kTile * D : kTileBytes;
    static constexpr int kKeys = D == 128 ? (I8 ? 4 : 3) : 6;
    static constexpr int kRawBytes = kTile * D;        // int8: value codes
    static constexpr int kRaws = !I8 ? 0 : D == 128 ? 4 : 6;
    static constexpr int kValues = D == 128 ? (I8 ? 2 : 3) : (I8 ? 4 : 6);
    static constexpr int kSmem = 1024 + kQBytes + 2 * kPBytes + kKeys * kKeyBytes +
                                 kRaws * kRawBytes + kValues * kTileBytes;
    static constexpr int kThreads = I8 ? 512 : 256;
    static constexpr uint32_t kColumns = I8 ? 256 : 128;  // tensor memory: S, S, O; codes
};

struct DecodeBars {
    uint64_t q_full, q_empty, key_full[6], key_empty[6], raw_full[6], raw_empty[6], value_full[6],
        value_empty[6], turned_full[2], turned_empty[2], s_full[2], p_full[2], o_done[2],
        done;
};

template <bool BF16, int D, int NR, bool I8>
__global__ void __launch_bounds__(DecodeShape<D, NR, I8>::kThreads, 1)
decode_paged_kernel(const __grid_constant__ DecodeArgs a, const __grid_constant__ CUtensorMap q_map,
                    const __grid_constant__ CUtensorMap k_map,
                    const __grid_constant__ CUtensorMap v_map) {
    using Sh = DecodeShape<D, NR, I8>;
    constexpr int kHalves = D / 64;
    constexpr int kHalfBytes = kTile * 128;
    constexpr int kRaws = I8 ? Sh::kRaws : 1;
    // int8: weights and value codes are f16 whatever the queries are (three more
    // bits, and the codes take fewer instructions)
    constexpr bool kPBf16 = BF16 && !I8;
    // above it a weight asks for a new reference (int8: weights are stored times up to 4)
    constexpr float kRedo = I8 ? 8192.0f : 32768.0f;

    extern __shared__ uint8_t raw_smem[];
    __shared__ DecodeBars bar;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag, last_piece;
    __shared__ uint32_t dead_groups[16];  // per key tile: its 16-key groups on bad pages
    __shared__ int tile_rows[16][8];      // int8, per key tile: its boxes' cache rows
    __shared__ float2 scales[I8 ? 4 : 1][kTile];  // and its keys' scales of keys and values
    __shared__ __align__(16) float m_s[NR], base_s[NR], f_s[NR];  // references, less or 0, to a new one
    __shared__ float red[4][NR], sums[4][NR];
    __shared__ uint32_t top_scale[4];  // int8: bits of the warps' largest value scales

    uint8_t *smem = raw_smem + ((1024 - (smem_addr(raw_smem) & 1023)) & 1023);
    uint8_t *q_smem = smem;
    uint8_t *p_smem = q_smem + Sh::kQBytes;
    uint8_t *keys = p_smem + 2 * Sh::kPBytes;
    uint8_t *raws = keys + Sh::kKeys * Sh::kKeyBytes;
    uint8_t *values = raws + Sh::kRaws * Sh::kRawBytes;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (warp == 6) tmem_alloc(&tmem_slot, Sh::kColumns);
    if (tid == 0) {
        mbar_init(&bar.q_full, 1);
        mbar_init(&bar.q_empty, 1);
        for (int i = 0; i < 6; ++i) {
            mbar_init(&bar.key_full[i], 1);
            mbar_init(&bar.key_empty[i], I8 ? 4 : 1);  // by the product, or who reads codes
            mbar_init(&bar.raw_full[i], 1);
            mbar_init(&bar.raw_empty[i], 4);
            mbar_init(&bar.value_full[i], I8 ? 4 : 1);
            mbar_init(&bar.value_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.turned_full[i], 4);
            mbar_init(&bar.turned_empty[i], 1);
            mbar_init(&bar.s_full[i], 1);
            mbar_init(&bar.p_full[i], 4);
            mbar_init(&bar.o_done[i], 1);
        }
        mbar_init(&bar.done, 2);
        fence_barrier_init();
        abort_flag = 0;
    }
    // rows that are none: zero queries
    for (int i = tid; i < Sh::kQBytes / 16; i += Sh::kThreads)
        reinterpret_cast<uint4 *>(q_smem)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async();
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    pdl_wait();
    pdl_launch_dependents();

    // ---- this CTA's piece of the line of key tiles, found by each warp
    auto cost_of = [&](int b, bool report) -> int {
        if (b >= a.c.batch) return 0;
        const Seq s = seq_of(a, b, report);
        return s.n > 0 ? run_of(a, s).tiles * a.c.n_kv_heads : 0;
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
    const int ctas = max(min(static_cast<int>(gridDim.x), total / a.min_tiles), 1);
    const int share = total / ctas, spare = total % ctas;
    auto cut = [&](int c) { return c * share + min(c, spare); };  // where CTA c begins
    // the CTA that holds tile x
    auto cta_of = [&](int x) {
        const int big = spare * (share + 1);
        return x < big ? x / (share + 1) : spare + (x - big) / max(share, 1);
    };
    Place w;
    w.left = 0;
    const int x0 = static_cast<int>(blockIdx.x) < ctas ? cut(blockIdx.x) : total;
    if (static_cast<int>(blockIdx.x) < ctas && total > 0) {
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
                w.s = seq_of(a, w.b, false);
                const int tiles = run_of(a, w.s).tiles;
                w.head = r / tiles;
                w.off = r - w.head * tiles;
                w.left = cut(blockIdx.x + 1) - x0;
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
    Run g;
    bool ok = true;
    constexpr uint32_t kOColumn = 2 * NR, kCodeColumn = 128;

    if (warp == 4 || warp == 5) {
        // ------------------------------------------------------------ loads ---
        const bool is_k = warp == 4;
        const uint64_t policy = l2_policy_evict_first();
        const int boxes = kTile / a.box, ps = a.c.page_size;
        const int per_read = 32 / boxes;  // tiles whose rows one read of the page table gives
        const int places = is_k ? Sh::kKeys : I8 ? kRaws : Sh::kValues;
        const int place_bytes = is_k ? Sh::kKeyBytes : I8 ? Sh::kRawBytes : Sh::kTileBytes;
        uint8_t *ring = is_k ? keys : I8 ? raws : values;
        uint64_t *full = is_k ? bar.key_full : I8 ? bar.raw_full : bar.value_full;
        uint64_t *empty = is_k ? bar.key_empty : I8 ? bar.raw_empty : bar.value_empty;
        const CUtensorMap *map = is_k ? &k_map : &v_map;
        uint32_t n = 0, st = 0, round = 0, queries = 0;  // queries: loads of them so far
#pragma unroll 1
        while (ok && next_run(a, w, g)) {
            if (is_k) {
                if (queries > 0 && !(ok = wait_for(&bar.q_empty, (queries - 1) & 1, abort))) break;
                ++queries;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&bar.q_full, a.max_new * a.G * 128 * kHalves);
                    for (int h = 0; h < kHalves; ++h)
                        tma_load_4d(q_smem + h * Sh::kQHalf, &q_map, h * 64, 0, g.head, g.s.s0,
                                    &bar.q_full);
                }
                __syncwarp();
            }
            // the cache rows of the boxes of tiles j, j + 1, .., a lane a box: dead_row
            // where none is needed, -1 on a bad page
            auto rows_of = [&](int j) -> int {
                const int t0 = (j + lane / boxes) * kTile + lane % boxes * a.box;
                if (t0 >= g.j1 * kTile || t0 >= g.hi || t0 + a.box <= g.lo) return a.dead_row;
                const int col = t0 / ps;
                const int page = checked_page(a.c, g.b, col);
                return page < 0 ? -1 : (page * a.c.n_kv_heads + g.head) * ps + (t0 - col * ps);
            };
            int rows = 0, rows_next = rows_of(g.j0);
#pragma unroll 1
            for (int j = g.j0; j < g.j1; ++j) {
                const int in = (j - g.j0) % per_read;
                if (in == 0) {
                    rows = rows_next;
                    rows_next = rows_of(j + per_read);
                }
                int row = __shfl_sync(0xffffffffu, rows, in * boxes + lane % boxes);
                const bool bad = row < 0;
                if (bad) row = a.dead_row;
                if (round > 0 && !(ok = wait_for(&empty[st], (round - 1) & 1, abort))) break;
                if (is_k) {
                    const int k = a.box / 16;
                    const uint32_t groups = __reduce_or_sync(
                        0xffffffffu, bad ? ((1u << k) - 1) << (lane % boxes * k) : 0u);
                    if (lane == 0) dead_groups[n & 15] = groups;
                    if (I8 && lane < boxes) tile_rows[n & 15][lane] = row;
                    __syncwarp();
                    if constexpr (I8) {
                        // The scales, which the turning warps read later, on their way to
                        // the L2: 16 tokens a lane, keys' and values'.  (8 sequences of
                        // 131,072 tokens, several caches in turn: 402 us without, 362.)
                        const int group = lane & 7;
                        const int box_row = __shfl_sync(0xffffffffu, row, group / k);
                        const float *sc = static_cast<const float *>(lane < 8 ? a.c.k_scale
                                                                              : a.c.v_scale);
                        if (lane < 16 && box_row != a.dead_row)
                            asm volatile("prefetch.global.L2 [%0];" ::"l"(
                                sc + box_row + group % k * 16));
                    }
                }
                if (lane == 0) mbar_arrive_expect_tx(&full[st], I8 ? kTile * D : Sh::kTileBytes);
                __syncwarp();
                uint8_t *dst = ring + st * place_bytes;
                if (lane < boxes) {
                    if constexpr (I8) {
                        tma_load_2d(dst + lane * a.box * D, map, 0, row, &full[st], policy);
                    } else {
#pragma unroll
                        for (int h = 0; h < kHalves; ++h)
                            tma_load_2d(dst + h * kHalfBytes + lane * a.box * 128, map, h * 64, row,
                                        &full[st], policy);
                    }
                }
                ++n;
                if (++st == static_cast<uint32_t>(places)) {
                    st = 0;
                    ++round;
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
            for (int i = 0; landed && i < places; ++i) {
                const uint32_t fills = round + (static_cast<uint32_t>(i) < st ? 1 : 0);
                if (fills > 0) landed = mbar_wait(&full[i], (fills - 1) & 1, &none);
            }
            if (landed && queries > 0) mbar_wait(&bar.q_full, (queries - 1) & 1, &none);
        }
        return;
    } else if (warp == 6) {
        // ------------------------------------------------- products S^T = K Q^T ---
        constexpr uint32_t kIdS = mma_idesc(BF16, kTile, NR, false);
        const uint32_t key_addr = smem_addr(keys);
        const uint32_t tmem_u = warp_uniform(tmem);
        const uint32_t q = warp_uniform(desc_low(smem_addr(q_smem), 16));
        uint32_t n = 0, st = 0, round = 0, q_phase = 0;
#pragma unroll 1
        while (ok && next_run(a, w, g)) {
            if (!(ok = wait_for(&bar.q_full, q_phase, abort))) break;
            q_phase ^= 1;
#pragma unroll 1
            for (int j = g.j0; j < g.j1; ++j, ++n) {
                const uint32_t b = n & 1;
                uint32_t k_at = 0, code = 0;
                if constexpr (I8) {
                    if (!(ok = wait_for(&bar.turned_full[b], (n >> 1) & 1, abort))) break;
                    code = warp_uniform(tmem_u + kCodeColumn + b * (D / 2));
                } else {
                    if (!(ok = wait_for(&bar.key_full[st], round & 1, abort))) break;
                    k_at = warp_uniform(desc_low(key_addr + st * Sh::kKeyBytes, 16));
                }
                // the logits of two tiles ago have been read, and their weights: what
                // the softmax needs to know to overwrite P comes with S
                if (n >= 2 && !(ok = wait_for(&bar.o_done[b], ((n >> 1) - 1) & 1, abort))) break;
                tmem_fence_after();
                const uint32_t s_at = warp_uniform(tmem_u + b * NR);
                if (elect_one()) {
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        const uint32_t in = (i % 4) * 32;
                        const uint64_t qd = smem_desc(q + ((i / 4) * Sh::kQHalf + in) / 16);
                        if constexpr (I8)
                            mma_ts(s_at, code + i * 8, qd, kIdS, i > 0);
                        else
                            mma_ss(s_at, smem_desc(k_at + ((i / 4) * kHalfBytes + in) / 16), qd,
                                   kIdS, i > 0);
                    }
                    mma_commit(&bar.s_full[b]);
                    mma_commit(I8 ? &bar.turned_empty[b] : &bar.key_empty[st]);
                    if (j + 1 == g.j1) mma_commit(&bar.q_empty);
                }
                __syncwarp();
                if (++st == Sh::kKeys) {
                    st = 0;
                    ++round;
                }
            }
        }
        if (!ok) fail();
        // every product and every barrier arrival is done before the CTA goes
        if (elect_one()) mma_commit(&bar.done);
        __syncwarp();
        volatile int none = 0;
        if (!mbar_wait(&bar.done, 0, &none)) fail();
    } else if (warp == 7) {
        // ---------------------------------------------- products O^T += V^T P^T ---
        constexpr uint32_t kIdO = mma_idesc(kPBf16, kTile, NR, false, true);
        const uint32_t value_addr = smem_addr(values);
        const uint32_t tmem_u = warp_uniform(tmem);
        uint32_t n = 0, st = 0, round = 0;
#pragma unroll 1
        while (ok && next_run(a, w, g)) {
#pragma unroll 1
            for (int j = g.j0; j < g.j1; ++j, ++n) {
                const uint32_t b = n & 1;
                if (!(ok = wait_for(&bar.value_full[st], round & 1, abort))) break;
                const int from = max(g.lo - j * kTile, 0), to = min(g.hi - j * kTile, kTile);
                if (!I8 && (from > 0 || to < kTile)) {
                    // value rows that no token sees may hold NaN: clear them
                    uint8_t *vs = values + st * Sh::kTileBytes;
                    const int c = (from + (kTile - max(to, 0))) * 8 * kHalves;
#pragma unroll 1
                    for (int i = lane; i < c; i += 32) {
                        int r = i / (8 * kHalves);
                        if (r >= from) r += max(to, 0) - from;
                        *reinterpret_cast<uint4 *>(vs + (i / 8) % kHalves * kHalfBytes + r * 128 +
                                                   i % 8 * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async();
                    __syncwarp();
                }
                if (!(ok = wait_for(&bar.p_full[b], (n >> 1) & 1, abort))) break;
                tmem_fence_after();
                // at D = 64 lanes 64 to 127 repeat the others
                const uint32_t v = warp_uniform(
                    desc_low(value_addr + st * Sh::kTileBytes, D == 128 ? kHalfBytes : 0));
                const uint32_t p = warp_uniform(desc_low(smem_addr(p_smem) + b * Sh::kPBytes, 16));
                const uint32_t add = warp_uniform(j > g.j0);
                if (elect_one()) {
#pragma unroll
                    for (int i = 0; i < kTile / 16; ++i)
                        mma_ss(tmem_u + kOColumn, smem_desc(v + i * (2048 / 16)),
                               smem_desc(p + ((i / 4) * (NR * 128) + (i % 4) * 32) / 16), kIdO,
                               i > 0 ? 1 : add);
                    mma_commit(&bar.value_empty[st]);
                    mma_commit(&bar.o_done[b]);
                }
                __syncwarp();
                if (++st == Sh::kValues) {
                    st = 0;
                    ++round;
                }
            }
        }
        if (!ok) fail();
        if (elect_one()) mma_commit(&bar.done);
        __syncwarp();
        volatile int none = 0;
        if (!mbar_wait(&bar.done, 0, &none)) fail();
    } else if (I8 && warp >= 8 && warp < 12) {
        // -------------------------------------- key codes to tensor memory ---
        const int row = tid - 256;  // the key, and the lane
        const uint32_t lanes = tmem + ((warp & 3) << 21) + kCodeColumn;
        const int swizzle = D == 128 ? row & 7 : (row >> 1) & 3;
        uint32_t n = 0, st = 0, round = 0;
#pragma unroll 1
        while (ok && next_run(a, w, g)) {
#pragma unroll 1
            for (int j = g.j0; j < g.j1; ++j) {
                if (!(ok = wait_for(&bar.key_full[st], round & 1, abort))) break;
                // this key's scales, on their way while its codes are turned
                const int cache_row = tile_rows[n & 15][row / a.box];
                const int tok = j * kTile + row;
                const bool live = cache_row != a.dead_row && tok >= g.lo && tok < g.hi;
                float2 sc = make_float2(0.0f, 0.0f);
                if (live) {
                    sc.x = static_cast<const float *>(a.c.k_scale)[cache_row + row % a.box];
                    sc.y = static_cast<const float *>(a.c.v_scale)[cache_row + row % a.box];
                }
                if (n >= 2 && !(ok = wait_for(&bar.turned_empty[n & 1], ((n >> 1) - 1) & 1, abort)))
                    break;
                tmem_fence_after();
                const uint8_t *src = keys + st * Sh::kKeyBytes + row * D;
#pragma unroll 1
                for (int c = 0; c < D / 16; c += 4) {
                    uint32_t o[32];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint4 x =
                            *reinterpret_cast<const uint4 *>(src + ((c + i) ^ swizzle) * 16);
                        codes_to<BF16>(x.x, o[8 * i], o[8 * i + 1]);
                        codes_to<BF16>(x.y, o[8 * i + 2], o[8 * i + 3]);
                        codes_to<BF16>(x.z, o[8 * i + 4], o[8 * i + 5]);
                        codes_to<BF16>(x.w, o[8 * i + 6], o[8 * i + 7]);
                    }
                    tmem_st32(lanes + (n & 1) * (D / 2) + c * 8, o);
                }
                scales[n & 3][row] = make_float2(sc.x * a.scale_log2, sc.y);
                tmem_wait_st();
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bar.turned_full[n & 1]);
                    mbar_arrive(&bar.key_empty[st]);
                }
                ++n;
                if (++st == Sh::kKeys) {
                    st = 0;
                    ++round;
                }
            }
        }
        if (!ok) fail();
    } else if (I8 && warp >= 12) {
        // ------------------------------------ value codes to shared memory ---
        // A lane's row and 16 codes of a step: the 8 lanes of a load or a store lie
        // on two rows, at D = 128 on the one's first half and the other's second, so
        // that the codes come from all banks; and as the swizzle turns even chunks of
        // an odd row into odd ones, the chunks go to all banks too.
        constexpr int kUnits = D / 16;          // 16-code steps a row
        constexpr int kRows = 32 / kUnits * 4;  // rows of a step of the four warps
        constexpr int kSteps = kTile / kRows;
        const int q8 = lane >> 3, k8 = lane & 7;
        const int row = (warp - 12) * (32 / kUnits) +
                        (D == 128 ? 2 * (q8 >> 1) + (k8 >> 2) : lane >> 2);
        const int u = D == 128 ? (k8 & 3) + 4 * ((q8 & 1) ^ (k8 >> 2)) : lane & 3;
        const int dst_row = (u / 4) * kHalfBytes + row * 128;
        const int dst0 = dst_row + 16 * (((u % 4) * 2) ^ (row & 7));
        const int dst1 = dst_row + 16 * (((u % 4) * 2 + 1) ^ (row & 7));
        static_assert(kRows % 8 == 0, "the swizzle of a lane's row stays");
        uint32_t st = 0, round = 0, v_st = 0, v_round = 0;
#pragma unroll 1
        while (ok && next_run(a, w, g)) {
#pragma unroll 1
            for (int j = g.j0; j < g.j1; ++j) {
                if (!(ok = wait_for(&bar.raw_full[st], round & 1, abort))) break;
                if (v_round > 0 &&
                    !(ok = wait_for(&bar.value_empty[v_st], (v_round - 1) & 1, abort)))
                    break;
                const uint8_t *src = raws + st * Sh::kRawBytes + row * D + 16 * u;
                uint8_t *dst = values + v_st * Sh::kTileBytes;
#pragma unroll 4
                for (int i = 0; i < kSteps; ++i) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(src + i * (kRows * D));
                    uint4 lo, hi;
                    codes_to<false>(x.x, lo.x, lo.y);
                    codes_to<false>(x.y, lo.z, lo.w);
                    codes_to<false>(x.z, hi.x, hi.y);
                    codes_to<false>(x.w, hi.z, hi.w);
                    *reinterpret_cast<uint4 *>(dst + dst0 + i * (kRows * 128)) = lo;
                    *reinterpret_cast<uint4 *>(dst + dst1 + i * (kRows * 128)) = hi;
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bar.value_full[v_st]);
                    mbar_arrive(&bar.raw_empty[st]);
                }
                if (++st == static_cast<uint32_t>(kRaws)) {
                    st = 0;
                    ++round;
                }
                if (++v_st == Sh::kValues) {
                    v_st = 0;
                    ++v_round;
                }
            }
        }
        if (!ok) fail();
    } else if (warp < 4) {
        // ------------------------------------------------------------ softmax ---
        const uint32_t lanes = tmem + (warp << 21);
        const int key = tid;
        uint32_t n = 0;
        int piece = 0;  // runs of this CTA so far
        int x = x0;
        // These warps meet at barriers of the hardware, which have no limit: so none
        // leaves its loops before the others, and a wait that ran out only makes the
        // waits behind it pass.
        auto wait = [&](uint64_t *b, uint32_t parity) {
            if (ok) ok = wait_for(b, parity, abort);
        };
#pragma unroll 1
        for (; next_run(a, w, g); ++piece) {
            const int rows = g.s.n * a.G;
            const int p0 = g.s.first;  // the first token's position
            // keys that every row sees
            const int all_lo = a.window > 0 ? max(p0 + g.s.n - a.window, 0) : 0;
            const int all_hi = max(p0 + 1, 0);
            float l[NR];
#pragma unroll
            for (int r = 0; r < NR; ++r) l[r] = 0.0f;
            ScaleUnit unit = {};  // int8
            bool open = true;   // a row has seen no key yet, and so has no reference
#pragma unroll 1
            for (int j = g.j0; j < g.j1; ++j, ++n) {
                const uint32_t b = n & 1;
                wait(&bar.s_full[b], (n >> 1) & 1);
                tmem_fence_after();
                const int t = j * kTile + key;
                const uint32_t bad = dead_groups[n & 15] >> (key / 16) & 1;
                float ks = a.scale_log2, vs = 1.0f;
                if constexpr (I8) {
                    const float2 sc = scales[n & 3][key];
                    ks = sc.x;
                    vs = sc.y;
                }
                // the rows that see this key
                uint32_t seen = 0xffffffffu;
                if (j * kTile < all_lo || (j + 1) * kTile > all_hi || bad) {
                    seen = 0;
                    if (t >= g.lo && t < g.hi && !bad) {
                        // of the tokens from t on, and with a window to t + window - 1
                        const int first = max(t - p0, 0);
                        int last = g.s.n - 1;
                        if (a.window > 0) last = min(last, t + a.window - 1 - p0);
                        if (first <= last) {
                            const int r0 = first * a.G, r1 = (last + 1) * a.G;  // r1 <= 32
                            seen = (r1 >= 32 ? 0xffffffffu : (1u << r1) - 1) & ~((1u << r0) - 1);
                        }
                    }
                }
                bool fix = open;
                float p[NR];
                float v;
#pragma unroll 1
                for (;;) {
                    float s[NR];
#pragma unroll
                    for (int i = 0; i < NR; i += 16) tmem_ld16(lanes + b * NR + i, s + i);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < NR; i += 16) pin16(s + i);
                    if (fix) {
                        // each row's maximum, over the warp's keys, then over all
                        float mine = -INFINITY;
#pragma unroll
                        for (int r = 0; r < NR; ++r) {
                            const uint32_t k = __reduce_max_sync(
                                0xffffffffu, float_to_key(seen >> r & 1 ? s[r] * ks : -INFINITY));
                            if (lane == r) mine = __uint_as_float(k);
                        }
                        if (lane < NR) red[warp][lane] = mine;
                        if constexpr (I8) {
                            const uint32_t u = __float_as_uint(vs);
                            const uint32_t top =
                                __reduce_max_sync(0xffffffffu, u < 0x7f800000u ? u : 0u);
                            if (lane == 0) top_scale[warp] = top;
                        }
                        // O as it stands is complete
                        if (j > g.j0) wait(&bar.o_done[b ^ 1], ((n - 1) >> 1) & 1);
                        meet_128();
                        const int old_exp = unit.exp;
                        if constexpr (I8)  // (the 2: weights times up to 4 fit f16)
                            unit.take(max(max(top_scale[0], top_scale[1]),
                                          max(top_scale[2], top_scale[3])),
                                      j == g.j0, 2);
                        bool none = false;
                        if (tid < NR) {
                            uint32_t k = 0;
#pragma unroll
                            for (int i = 0; i < 4; ++i) k = max(k, __float_as_uint(red[i][tid]));
                            const float top = key_to_float(k);
                            const float m = j == g.j0 ? -INFINITY : m_s[tid];
                            const float mn = fmaxf(m, top - kLift);
                            f_s[tid] = m == -INFINITY || mn == -INFINITY ? 1.0f : exp2_approx(m - mn);
                            m_s[tid] = mn;
                            none = tid < rows && mn == -INFINITY;
                            // rows that are none (another sequence's queries may stand
                            // there): no weights, and no say in the votes
                            base_s[tid] = tid >= rows      ? -INFINITY
                                          : mn == -INFINITY ? 0.0f
                                                            : -mn;
                        }
                        open = any_of_128(none);
                        // up by at most 2^60 (ScaleUnit), down to 0 where it matters
                        const float fu =
                            I8 ? exp2_approx(static_cast<float>(old_exp - unit.exp)) : 1.0f;
#pragma unroll
                        for (int r = 0; r < NR; ++r) l[r] *= f_s[r];
                        if (j > g.j0) {
                            tmem_fence_after();
#pragma unroll 1
                            for (int i = 0; i < NR; i += 16) {
                                float o[16];
                                tmem_ld16(lanes + kOColumn + i, o);
                                tmem_wait_ld();
                                pin16(o);
#pragma unroll
                                for (int r = 0; r < 16; ++r) o[r] *= f_s[i + r] * fu;
                                tmem_st16(lanes + kOColumn + i, reinterpret_cast<uint32_t *>(o));
                            }
                            tmem_wait_st();
                            tmem_fence_before();
                        }
                    }
                    v = I8 ? vs * __int_as_float((127 - unit.exp) << 23) : 1.0f;
                    const float2 k2 = make_float2(ks, ks);
                    float top = 0.0f;
#pragma unroll
                    for (int r = 0; r < NR; r += 4) {
                        const float4 base = *reinterpret_cast<const float4 *>(base_s + r);
                        const float2 u0 = __ffma2_rn(make_float2(s[r], s[r + 1]), k2,
                                                     make_float2(base.x, base.y));
                        const float2 u1 = __ffma2_rn(make_float2(s[r + 2], s[r + 3]), k2,
                                                     make_float2(base.z, base.w));
                        p[r] = exp2_approx(u0.x);
                        p[r + 1] = exp2_approx(u0.y);
                        p[r + 2] = exp2_approx(u1.x);
                        p[r + 3] = exp2_approx(u1.y);
                    }
                    if (seen != 0xffffffffu)
#pragma unroll
                        for (int r = 0; r < NR; ++r)
                            if (!(seen >> r & 1)) p[r] = 0.0f;
#pragma unroll
                    for (int r = 0; r < NR; r += 2) top = fmax3(top, p[r], p[r + 1]);
                    if (fix) break;  // no weight passes 2^kLift
                    // int8: a new unit too, where a scale does not fit, or a warp's are
                    // so small that the unit may have to fall
                    const bool low = I8 && !__any_sync(0xffffffffu, v >= 0x1p-6f) &&
                                     __any_sync(0xffffffffu, v > 0.0f);
                    if (!any_of_128(top > kRedo || (I8 && v > 4.0f) || low)) break;
                    fix = true;
                }
                // the weights, and P^T: row r's 128 keys in two swizzled halves
                uint8_t *dst = p_smem + b * Sh::kPBytes + (key / 64) * (NR * 128) + (key % 8) * 2;
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    l[r] += p[r];
                    const float x = I8 ? p[r] * v : p[r];
                    *reinterpret_cast<uint16_t *>(dst + r * 128 +
                                                  (((key % 64) / 8) ^ (r & 7)) * 16) =
                        static_cast<uint16_t>(pack2<kPBf16>(x, 0.0f));
                }
                fence_proxy_async();
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.p_full[b]);
            }
            // ---- the run's sums
#pragma unroll
            for (int r = 0; r < NR; ++r) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
            }
            float mine = 0.0f;
#pragma unroll
            for (int r = 0; r < NR; ++r)
                if (lane == r) mine = l[r];
            if (lane < NR) sums[warp][lane] = mine;
            wait(&bar.o_done[(n - 1) & 1], ((n - 1) >> 1) & 1);
            tmem_fence_after();
            meet_128();
            float sum = 0.0f, m = -INFINITY;  // of row `lane`
            if (lane < NR) {
                sum = (sums[0][lane] + sums[1][lane]) + (sums[2][lane] + sums[3][lane]);
                m = m_s[lane];
            }
            float o[NR];
#pragma unroll
            for (int i = 0; i < NR; i += 16) tmem_ld16(lanes + kOColumn + i, o + i);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < NR; i += 16) pin16(o + i);
            const bool channel = key < D;
            const bool whole = g.off == 0 && g.j1 - g.j0 == g.tiles;
            const float out_unit = I8 ? __int_as_float((127 + unit.exp) << 23) : 1.0f;
            uint16_t *out = a.out + static_cast<int64_t>(g.s.s0) * a.out_stride +
                            static_cast<int64_t>(g.head) * a.G * D + key;
            const float inv = sum > 0.0f || sum != sum ? out_unit / sum : 0.0f;
            const uint32_t slot = 2 * blockIdx.x + (piece == 0 ? 0 : 1);
            auto write = [&](int r, float x) {  // channel `key` of row r
                const int tok = r / a.G;
                out[tok * a.out_stride + (r - tok * a.G) * D] =
                    static_cast<uint16_t>(pack2<BF16>(x, 0.0f));
            };
            if (whole) {
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const float f = __shfl_sync(0xffffffffu, inv, r);
                    if (channel && r < rows) write(r, f != 0.0f ? o[r] * f : 0.0f);
                }
            } else {
                if (warp == 0 && lane < rows) a.ml[slot * NR + lane] = make_float2(m, sum);
#pragma unroll
                for (int r = 0; r < NR; ++r)
                    if (channel && r < rows) a.acc[(slot * NR + r) * D + key] = o[r] * out_unit;
                // the last of the item's CTAs to arrive joins them
                const int begin = x - g.off, end = begin + g.tiles;
                const int c0 = max(cta_of(begin), 0), c1 = min(cta_of(end - 1), ctas - 1);
                __threadfence();
                meet_128();
                if (tid == 0) {
                    const unsigned was = atomic_add_acq_rel_gpu(&a.arrived[c0], 1u);
                    last_piece = was == static_cast<unsigned>(c1 - c0);
                    if (last_piece) a.arrived[c0] = 0;
                }
                meet_128();
                if (last_piece) {
                    __threadfence();
                    // CTA c0's piece is its last run, the others' their first
                    const uint32_t first_slot = 2 * c0 + (cut(c0) < begin ? 1 : 0);
                    auto slot_of = [&](int c) { return c == c0 ? first_slot : 2u * c; };
                    // The pieces' factors, a warp a row and a lane a piece, for half of the
                    // rows at a time where P was (read already: the run's last product is
                    // done); then the sums, a thread a channel with 32 reads under way.
                    constexpr int kRowsAt = 2 * Sh::kPBytes / (kMaxCtas * 4);
                    float *factors = reinterpret_cast<float *>(p_smem);
#pragma unroll 1
                    for (int r0 = 0; r0 < rows; r0 += kRowsAt) {
                        const int r1 = min(r0 + kRowsAt, rows);
                        if (r0 > 0) meet_128();
#pragma unroll 1
                        for (int r = r0 + warp; r < r1; r += 4) {
                            float top = -INFINITY, den = 0.0f;
                            for (int c = c0 + lane; c <= c1; c += 32)
                                top = fmaxf(top, __ldcg(&a.ml[slot_of(c) * NR + r]).x);
#pragma unroll
                            for (int o = 16; o > 0; o >>= 1)
                                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                            for (int c = c0 + lane; c <= c1; c += 32) {
                                const float2 ml = __ldcg(&a.ml[slot_of(c) * NR + r]);
                                const float f = ml.x == -INFINITY ? 0.0f : exp2_approx(ml.x - top);
                                den = fmaf(f, ml.y, den);
                                factors[(r - r0) * kMaxCtas + c - c0] = f;
                            }
#pragma unroll
                            for (int o = 16; o > 0; o >>= 1)
                                den += __shfl_xor_sync(0xffffffffu, den, o);
                            if (lane == 0) sums[0][r] = den > 0.0f || den != den ? 1.0f / den : 0.0f;
                        }
                        meet_128();
                        if (channel)
#pragma unroll 1
                            for (int r = r0; r < r1; r += 4) {
                                float o[4] = {};
#pragma unroll 1
                                for (int c = c0; c <= c1; c += 8) {
                                    float u[4][8];
#pragma unroll
                                    for (int q = 0; q < 4; ++q)
                                        if (r + q < r1)
#pragma unroll
                                            for (int i = 0; i < 8; ++i)
                                                if (c + i <= c1)
                                                    u[q][i] = __ldcg(
                                                        &a.acc[(slot_of(c + i) * NR + r + q) * D + key]);
#pragma unroll
                                    for (int q = 0; q < 4; ++q)
                                        if (r + q < r1)
#pragma unroll
                                            for (int i = 0; i < 8; ++i)
                                                if (c + i <= c1) {
                                                    const float f = factors[(r + q - r0) * kMaxCtas +
                                                                            c + i - c0];
                                                    if (f != 0.0f) o[q] = fmaf(f, u[q][i], o[q]);
                                                }
                                }
#pragma unroll
                                for (int q = 0; q < 4; ++q)
                                    if (r + q < r1) write(r + q, o[q] * sums[0][r + q]);
                            }
                    }
                    meet_128();           // the next tile's P goes there
                    fence_proxy_async();
                }
            }
            x += g.j1 - g.j0;
        }
        if (!ok) fail();
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == 6) {
        tmem_fence_after();
        tmem_free(tmem, Sh::kColumns);
    }
}

struct DecodePlan {
    int ctas;
    size_t ml, acc, total;
};

DecodePlan plan_of(int rows, int D) {
    DecodePlan w;
    w.ctas = device_sm_count() < kMaxCtas ? device_sm_count() : kMaxCtas;
    const size_t nr = rows <= 16 ? 16 : 32;
    w.ml = paged_counter_bytes();
    w.acc = w.ml + (w.ctas * 2 * nr * sizeof(float2) + 255) / 256 * 256;
    w.total = w.acc + (w.ctas * 2 * nr * D * sizeof(float) + 255) / 256 * 256;
    return w;
}

template <bool BF16, int D, int NR, bool I8>
cudaError_t launch_shape(const PagedAttnArgs &p, void *ws, cudaStream_t st) {
    using Sh = DecodeShape<D, NR, I8>;
    DecodeArgs a = {};
    CUtensorMap q_map, k_map, v_map;
    constexpr CUtensorMapSwizzle k_swizzle = I8 && D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                           : CU_TENSOR_MAP_SWIZZLE_128B;
    constexpr CUtensorMapSwizzle v_swizzle =
        I8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B;
    if (!fill_launch(p, p.max_new, k_swizzle, v_swizzle, a, q_map, k_map, v_map))
        return cudaErrorInvalidValue;
    const DecodePlan w = plan_of(p.max_new * p.G, D);
    // Shorter pieces cost more in joining than they mostly save: at 2, 4 and 6 tiles a
    // CTA at least one token over 512, 1024, 4096 and 8192 tokens took 9.8, 10.4, 12.0
    // and 15.6 us, 8.2, 11.3, 12.3 and 13.2, and 16.7, 15.5, 15.3 and 16.5.
    a.min_tiles = 4;
    uint8_t *base = static_cast<uint8_t *>(ws);
    a.arrived = reinterpret_cast<uint32_t *>(base);
    a.ml = reinterpret_cast<float2 *>(base + w.ml);
    a.acc = reinterpret_cast<float *>(base + w.acc);
    auto *kernel = decode_paged_kernel<BF16, D, NR, I8>;
    cudaError_t e =
        prepare_kernel(reinterpret_cast<const void *>(kernel), Sh::kThreads, Sh::kSmem);
    if (e != cudaSuccess) return e;
    return launch_ex(kernel, dim3(w.ctas), dim3(Sh::kThreads), Sh::kSmem, st, true, a, q_map, k_map,
                     v_map);
}

template <bool BF16, bool I8>
cudaError_t launch_type(const PagedAttnArgs &p, void *ws, cudaStream_t st) {
    // 16 rows take half the logits and weights of 32: one token of 4 heads over an int8
    // cache (4 sequences of 32,000) 67 us against 97, f16 over 512 tokens 8.2 against 10.3
    const bool narrow = p.max_new * p.G <= 16;
    if (p.c.head_dim == 64)
        return narrow ? launch_shape<BF16, 64, 16, I8>(p, ws, st)
                      : launch_shape<BF16, 64, 32, I8>(p, ws, st);
    return narrow ? launch_shape<BF16, 128, 16, I8>(p, ws, st)
                  : launch_shape<BF16, 128, 32, I8>(p, ws, st);
}

}  // namespace

size_t paged_counter_bytes() {
    return (device_sm_count() * sizeof(uint32_t) + 255) / 256 * 256;
}

size_t paged_decode_ws(int rows, int D) { return plan_of(rows, D).total; }

cudaError_t launch_paged_decode(const PagedAttnArgs &a, void *ws, cudaStream_t st) {
    if (a.c.dtype == KVD_INT8)
        return a.bf16 ? launch_type<true, true>(a, ws, st) : launch_type<false, true>(a, ws, st);
    return a.bf16 ? launch_type<true, false>(a, ws, st) : launch_type<false, false>(a, ws, st);
}

}  // namespace kvd
