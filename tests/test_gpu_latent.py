"""kvd_latent_append and kvd_latent_attn against 64-bit references (bounds in latent_ref.py)."""
import math

import pytest
import torch

import latent_ref as LR
import long_context_decode_kv_gb300 as kvd
import paged_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
X = {kvd.F16: torch.float16, kvd.BF16: torch.bfloat16}


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _starts(new):
    return torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int32, device=DEV)


def _cache(dtype, lens, page, seed, rank=512, rope_dim=64, spare=1):
    """A cache of scattered pages that hold data in every row (stale ones too)."""
    B = len(lens)
    cols = max(1, max((n + page - 1) // page for n in lens)) + spare
    c = kvd.LatentCache(dtype, B, B * cols, page, cols, rank=rank, rope_dim=rope_dim)
    c.page_table.copy_(R.scattered_tables(B, cols, seed, DEV))
    c.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
    c.len = max(lens)
    c.rows.copy_(torch.randn(c.rows.shape, generator=_gen(seed), device=DEV))
    return c


def _q(T, H, D, x, seed, scale=1.0):
    return (torch.randn(T, H, D, generator=_gen(seed), device=DEV) * scale).to(x)


def _attend(c, q, new, window=0, scale=0.07, ws=None, max_new=None, lse=True):
    T, H, _ = q.shape
    out = torch.full((T, H, c.rank), math.nan, device=DEV, dtype=q.dtype)
    lse = torch.full((T, H), math.nan, device=DEV) if lse else None
    max_new = max_new or max(new)
    ws = kvd.make_latent_workspace(c, H, T, max_new) if ws is None else ws
    kvd.latent_attn(c, q, _starts(new), max_new, scale, out, ws, window=window, lse=lse)
    return out, lse


def _check(c, q, new, window=0, scale=0.07, **kw):
    out, lse = _attend(c, q, new, window, scale, **kw)
    assert c.device_status() == 0
    want = LR.attn(c, q, _starts(new).tolist(), c.seq_lens.tolist(), scale, window)
    LR.assert_close(out, want["out"], "out")
    LR.assert_close(lse, want["lse"], "lse")
    n = sum(new)
    assert out[n:].isnan().all() and lse[n:].isnan().all()    # rows of no sequence
    return out, lse


# ----------------------------------------------------------------- append ---

@pytest.mark.parametrize("dtype", [kvd.F16, kvd.BF16])
@pytest.mark.parametrize("x", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page,rank,P,rot,H,inter,norm", [
    (16, 512, 64, 64, 5, False, True), (48, 128, 32, 16, 16, True, False),
    (64, 384, 48, 48, 1, False, True), (256, 256, 16, 16, 130, True, True)])
def test_append(dtype, x, page, rank, P, rot, H, inter, norm):
    new, lens = [5, 0, 1, 130, 17], [5, 40, 65, 200, 400]
    T = sum(new) + 3                                  # three padding rows behind the last sequence
    c = _cache(dtype, lens, page, page + rank, rank, P)
    before = c.rows.clone()
    g = _gen(3)
    down = (torch.randn(T, rank + P, generator=g, device=DEV) * 3).to(x)
    lat, k_pe = down[:, :rank], down[:, rank:]
    q_pe = torch.randn(T, H, 32 + P, generator=g, device=DEV).to(x)[:, :, 32:]
    w = torch.rand(rank, generator=g, device=DEV) + 0.5 if norm else None
    q_out = torch.full((T, H, rank + P), 7.0, device=DEV, dtype=x)
    rope = kvd.rope_table(rot, interleaved=inter, scaling="yarn", factor=4, orig_len=4096)
    kvd.latent_append(c, lat, k_pe, _starts(new), rope=rope, c_weight=w, q_pe=q_pe, q_out=q_out)
    assert c.device_status() == 0
    f, m = R.freqs(rot, 10000.0, "yarn", 4, 4096)
    n = sum(new)
    pos = torch.cat([torch.arange(l - k, l) for k, l in zip(new, lens)]).to(DEV)
    seq = torch.cat([torch.full((k,), b) for b, k in enumerate(new)]).to(DEV)
    page_of, in_page = c.page_table[seq, pos // page].long(), pos % page
    got = c.rows[page_of, in_page]
    y, err = R.turned(lat[:n, None], pos, None, 1.0, inter, w)
    R.assert_within(got[:, :rank], y[:, 0], R.rounding(y, err, X[dtype])[:, 0], "latent")
    y, err = R.turned(k_pe[:n, None], pos, f, m, inter)
    R.assert_within(got[:, rank:], y[:, 0], R.rounding(y, err, X[dtype])[:, 0], "key part")
    y, err = R.turned(q_pe[:n], pos, f, m, inter)
    R.assert_within(q_out[:n, :, rank:], y, R.rounding(y, err, x), "q")
    assert torch.all(q_out[n:] == 7.0) and torch.all(q_out[:, :, :rank] == 7.0)
    keep = torch.ones(c.n_pages, page, dtype=torch.bool, device=DEV)
    keep[page_of, in_page] = False
    assert torch.equal(c.rows[keep], before[keep])


def test_append_without_rotation_or_norm_copies():
    c = _cache(kvd.BF16, [40, 9], 16, 1, 128, 32)
    lat, k = _q(12, 1, 128, torch.bfloat16, 2)[:, 0], _q(12, 1, 32, torch.bfloat16, 3)[:, 0]
    kvd.latent_append(c, lat, k, _starts([3, 9]))
    pages = c.page_table.tolist()
    for t in range(12):
        b, p = (0, 37 + t) if t < 3 else (1, t - 3)
        row = c.rows[pages[b][p // 16], p % 16]
        assert torch.equal(row, torch.cat([lat[t], k[t]]))
    q = _q(12, 3, 160, torch.bfloat16, 4)
    was = q.clone()
    kvd.latent_append(c, lat, k, _starts([3, 9]), q_pe=q[:, :, 128:], q_out=q)    # in place
    assert torch.equal(q, was)


def test_append_checks_what_the_device_holds():
    def fresh():
        c = _cache(kvd.F16, [20, 20, 20], 16, 5, 128, 16)
        return c, _q(12, 1, 128, torch.float16, 6)[:, 0], _q(12, 1, 16, torch.float16, 7)[:, 0], c.rows.clone()

    for bad in (-1, 10 ** 6):
        c, x, k, before = fresh()
        c.page_table[1, 1] = bad
        kvd.latent_append(c, x, k, _starts([4, 4, 4]))
        assert c.device_status() == 1
        changed = (c.rows != before).any(-1)
        assert int(changed.sum()) == 8
        for b in (0, 2):
            assert changed[int(c.page_table[b, 1]), :4].all()
    c, x, k, before = fresh()
    c.seq_lens[1] = 2                                           # four new tokens in a length of two
    kvd.latent_append(c, x, k, _starts([4, 4, 4]))
    assert c.device_status() == 1
    changed = (c.rows != before).any(-1)
    assert int(changed.sum()) == 10 and changed[int(c.page_table[1, 0]), :2].all()


# -------------------------------------------------------------- attention ---

@pytest.mark.parametrize("dtype", [kvd.F16, kvd.BF16])
@pytest.mark.parametrize("H", [1, 3, 16, 20, 32, 48, 64, 65, 100, 128, 130])
def test_single_tokens(dtype, H):
    lens = [1, 7, 63, 64, 65, 300, 1029]
    c = _cache(dtype, lens, 64, H)
    _check(c, _q(len(lens), H, 576, X[dtype], H + 1), [1] * len(lens))


@pytest.mark.parametrize("dtype", [kvd.F16, kvd.BF16])
@pytest.mark.parametrize("rank,P", [(128, 16), (128, 64), (256, 32), (384, 48), (512, 64), (512, 16)])
@pytest.mark.parametrize("page", [16, 48, 128])
def test_ragged_batches(dtype, rank, P, page):
    """Chunks, single tokens, a sequence without a new token, padding rows."""
    new, lens = [1, 70, 0, 5, 33, 1, 129], [130, 70, 50, 400, 33, 777, 200]
    H = 12
    c = _cache(dtype, lens, page, page + rank, rank, P)
    _check(c, _q(sum(new) + 2, H, rank + P, X[dtype], 5), new)


@pytest.mark.parametrize("H,new", [(128, 3), (64, 9), (24, 40), (7, 100), (2, 150), (16, 4), (16, 3), (8, 4)])
@pytest.mark.parametrize("window", [0, 1, 50, 64, 500])
def test_chunks_and_windows(H, new, window):
    lens = [new + 400, new, new + 63]
    c = _cache(kvd.BF16, lens, 32, H + new, 256, 32)
    _check(c, _q(3 * new, H, 288, torch.bfloat16, 8), [new] * 3, window=window)


@pytest.mark.parametrize("dtype", [kvd.F16, kvd.BF16])
def test_long_contexts_cut_between_ctas(dtype):
    lens = [20000, 9, 33001]
    c = _cache(dtype, lens, 64, 3)
    q = _q(3, 40, 576, X[dtype], 4)
    out, lse = _check(c, q, [1, 1, 1])
    for _ in range(3):                                   # the same bits each time
        again, lse2 = _attend(c, q, [1, 1, 1])
        assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_lse_does_not_change_the_output():
    c = _cache(kvd.F16, [3000, 500], 64, 3)
    q = _q(40, 16, 576, torch.float16, 4)
    assert torch.equal(_attend(c, q, [20, 20])[0], _attend(c, q, [20, 20], lse=False)[0])


def test_many_sequences():
    B = 700
    lens = [1 + (b * 37) % 130 for b in range(B)]
    new = [min(b % 4, lens[b]) for b in range(B)]
    new[5], lens[5] = 90, 400
    c = _cache(kvd.BF16, lens, 16, 8, 128, 32)
    _check(c, _q(sum(new), 6, 160, torch.bfloat16, 9), new)


def test_rising_logits_move_the_reference():
    """Each tile's logits pass the ones before by far: the reference rises, O is scaled."""
    for dtype in (kvd.F16, kvd.BF16):
        c = _cache(dtype, [1000], 64, 2)
        q = _q(4, 16, 576, X[dtype], 3)
        ramp = torch.linspace(0.1, 4.0, 1000, device=DEV)
        for p in range((1000 + 63) // 64):
            n = min(64, 1000 - 64 * p)
            rows = c.rows[int(c.page_table[0, p]), :n].double()
            rows = rows * ramp[64 * p:64 * p + n, None]
            c.rows[int(c.page_table[0, p]), :n] = rows.to(X[dtype])
        _check(c, q, [4], scale=0.3)


def test_one_heavy_key_leaves_the_small_weights():
    c = _cache(kvd.F16, [3000], 64, 2)
    q = _q(1, 16, 576, torch.float16, 3)
    c.rows[int(c.page_table[0, 0]), 0] = q[0, 0] * 0.4
    _check(c, q, [1], scale=0.05)


def test_stale_rows_and_neighbours_do_not_count():
    """NaN in rows behind a length, in pages nobody needs, in another sequence's queries."""
    lens, new = [65, 130, 10], [2, 40, 10]
    c = _cache(kvd.BF16, lens, 16, 2)
    q = _q(sum(new), 16, 576, torch.bfloat16, 3)
    want, want_lse = _attend(c, q, new)
    used = torch.zeros(c.n_pages, 16, dtype=torch.bool, device=DEV)
    for b, l in enumerate(lens):
        for t in range(l):
            used[int(c.page_table[b, t // 16]), t % 16] = True
    c.rows[~used] = math.nan
    out, lse = _attend(c, q, new)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    q[2:42] = math.nan                                    # the middle sequence's own queries
    out, lse = _attend(c, q, new)
    keep = torch.ones(sum(new), dtype=torch.bool, device=DEV)
    keep[2:42] = False
    assert torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], want_lse[keep])
    assert out[2:42].isnan().all()
    assert c.device_status() == 0


def test_hidden_rows_may_hold_anything():
    """A window hides the first keys of all rows: infinities there do not count."""
    c = _cache(kvd.BF16, [300], 16, 2)
    q = _q(5, 16, 576, torch.bfloat16, 3)
    want, _ = _attend(c, q, [5], window=37)
    hidden = [t for t in range(300 - 5 - 37 + 1)]     # up to the middle of a tile
    for t in hidden:
        c.rows[int(c.page_table[0, t // 16]), t % 16] = math.inf
    out, _ = _attend(c, q, [5], window=37)
    assert torch.equal(out, want)


def test_rows_without_keys():
    """More new tokens than the length: those before position 0 see nothing, and it is reported."""
    c = _cache(kvd.F16, [3, 100], 16, 2)
    q = _q(9, 16, 576, torch.float16, 3)
    out, lse = _attend(c, q, [5, 4])
    assert c.device_status() == 1
    assert torch.all(out[:2] == 0) and torch.all(lse[:2] == -math.inf)
    want = LR.attn(c, q[2:], [0, 3, 7], [3, 100], 0.07)
    LR.assert_close(out[2:], want["out"])
    LR.assert_close(lse[2:], want["lse"])


def test_bad_pages_are_left_out():
    c = _cache(kvd.F16, [200, 200], 16, 2)
    q = _q(2, 16, 576, torch.float16, 3)
    good, _ = _attend(c, q, [1, 1])
    for bad in (-1, c.n_pages, 1 << 30):
        c.t["status"].zero_()
        t = c.page_table.clone()
        c.page_table[0, 3] = bad
        out, lse = _attend(c, q, [1, 1])
        assert c.device_status() == 1
        assert torch.equal(out[1], good[1])
        c.page_table.copy_(t)
        short = _cache(kvd.F16, [184], 16, 2)
        keep = [t for t in range(200) if not 48 <= t < 64]
        for i, s in enumerate(keep):
            short.rows[int(short.page_table[0, i // 16]), i % 16] = c.rows[int(t[0, s // 16]), s % 16]
        want = LR.attn(short, q[:1], [0, 1], [184], 0.07)
        LR.assert_close(out[:1], want["out"])
        LR.assert_close(lse[:1], want["lse"])


def test_strided_queries_and_outputs():
    c = _cache(kvd.F16, [300, 90], 64, 2)
    q = _q(50, 24, 576, torch.float16, 3)
    wide = torch.zeros(50, 40, 576, dtype=torch.float16, device=DEV)
    wide[:, 8:32] = q
    out = torch.full((50, 30, 512), 7.0, dtype=torch.float16, device=DEV)
    ws = kvd.make_latent_workspace(c, 24, 50, 40)
    kvd.latent_attn(c, wide[:, 8:32], _starts([10, 40]), 40, 0.07, out[:, 2:26], ws)
    want, _ = _attend(c, q, [10, 40])
    assert torch.equal(out[:, 2:26], want)
    assert torch.all(out[:, :2] == 7.0) and torch.all(out[:, 26:] == 7.0)


def test_one_workspace_for_calls_of_every_length():
    c = _cache(kvd.BF16, [5000, 300], 64, 2)
    ws = kvd.make_latent_workspace(c, 64, 600, 300)
    ws.random_(0, 256)                                   # needs no zeros
    for new in ([1, 1], [300, 300], [2, 7], [1, 0], [40, 300]):
        _check(c, _q(sum(new), 64, 576, torch.bfloat16, 3), new, ws=ws, max_new=300)
        _check(c, _q(sum(new), 64, 576, torch.bfloat16, 3), new, ws=ws)


def test_captured_and_on_another_stream():
    c = _cache(kvd.F16, [700, 64], 64, 2)
    q = _q(2, 32, 576, torch.float16, 3)
    want, want_lse = _attend(c, q, [1, 1])
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    ws = kvd.make_latent_workspace(c, 32, 2, 1)
    starts = _starts([1, 1])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    kvd.latent_attn(c, q, starts, 1, 0.07, out, ws, lse=lse, stream=side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvd.latent_attn(c, q, starts, 1, 0.07, out, ws, lse=lse)
    out.zero_()
    c.rows.mul_(0.5)
    c.seq_lens[0] = 650
    graph.replay()
    torch.cuda.synchronize()
    want, want_lse = _attend(c, q, [1, 1])
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_decode_steps_as_a_server_runs_them():
    """Append and attend, token after token, against a reference that keeps the rows itself."""
    H, rank, P = 8, 256, 32
    c = _cache(kvd.BF16, [40, 90], 16, 2, rank, P, spare=3)
    rope = kvd.rope_table(P, 10000.0)
    ws = kvd.make_latent_workspace(c, H, 2, 1)
    g = _gen(6)
    for step in range(20):
        c.seq_lens += 1
        c.len = c.len + 1
        lat = torch.randn(2, rank, generator=g, device=DEV).bfloat16()
        k_pe = torch.randn(2, P, generator=g, device=DEV).bfloat16()
        q = torch.randn(2, H, rank + P, generator=g, device=DEV).bfloat16()
        q_pe = q[:, :, rank:].clone()
        w = torch.ones(rank, device=DEV)
        kvd.latent_append(c, lat, k_pe, _starts([1, 1]), rope=rope, c_weight=w, q_pe=q_pe, q_out=q)
        out = torch.empty(2, H, rank, device=DEV, dtype=torch.bfloat16)
        kvd.latent_attn(c, q, _starts([1, 1]), 1, 0.08, out, ws)
        want = LR.attn(c, q, [0, 1, 2], c.seq_lens.tolist(), 0.08)
        LR.assert_close(out, want["out"], f"step {step}")
    assert c.device_status() == 0


def test_rows_before_the_first_sequence_and_runs_longer_than_told():
    c = _cache(kvd.F16, [90, 300], 16, 2)
    q = _q(40, 16, 576, torch.float16, 3)
    starts = torch.tensor([3, 13, 33], dtype=torch.int32, device=DEV)
    out = torch.full((40, 16, 512), 7.0, device=DEV, dtype=torch.float16)
    lse = torch.full((40, 16), 7.0, device=DEV)
    ws = kvd.make_latent_workspace(c, 16, 40, 20)
    kvd.latent_attn(c, q, starts, 20, 0.07, out, ws, lse=lse)
    assert c.device_status() == 0
    want = LR.attn(c, q, starts.tolist(), [90, 300], 0.07)
    LR.assert_close(out, want["out"])
    LR.assert_close(lse, want["lse"])
    rest = [0, 1, 2] + list(range(33, 40))
    assert torch.all(out[rest] == 7.0) and torch.all(lse[rest] == 7.0)
    out.fill_(7.0)
    kvd.latent_attn(c, q, starts, 12, 0.07, out, ws)              # the second run has 20: 12 are served
    assert c.device_status() == 1
    LR.assert_close(out[:25], (want["out"][0][:25], want["out"][1][:25]))
    assert torch.all(out[25:] == 7.0)


def test_an_empty_cache():
    c = _cache(kvd.BF16, [1, 1], 16, 2)
    c.seq_lens.zero_()
    c.len = 0
    q = _q(2, 16, 576, torch.bfloat16, 3)
    out, lse = _attend(c, q, [1, 1])
    assert c.device_status() == 1                                # a token needs a length of one
    assert torch.all(out == 0) and torch.all(lse == -math.inf)


@pytest.mark.parametrize("H", [300, 1024])
def test_many_heads(H):
    c = _cache(kvd.BF16, [100, 700], 64, 2, 128, 16)
    _check(c, _q(5, H, 144, torch.bfloat16, 3), [1, 4])


def test_two_streams_at_once():
    """Calls on two caches, each with its workspace, at the same time."""
    caches = [_cache(kvd.F16, [9000, 500], 64, i) for i in (2, 3)]
    qs = [_q(2, 64, 576, torch.float16, i) for i in (4, 5)]
    want = [_attend(c, q, [1, 1]) for c, q in zip(caches, qs)]
    ws = [kvd.make_latent_workspace(c, 64, 2, 1) for c in caches]
    outs = [torch.empty_like(w[0]) for w in want]
    starts = _starts([1, 1])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, q, w, o, s in zip(caches, qs, ws, outs, streams):
            kvd.latent_attn(c, q, starts, 1, 0.07, o, w, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w[0])


def test_offsets_above_32_bits():
    """Pages at the end of a pool of more than 2^32 bytes (and 2^31 elements)."""
    page, rank, P = 256, 512, 64
    n_pages = (1 << 32) // (page * 576) + 40
    rows = torch.empty(n_pages, page, rank + P, dtype=torch.bfloat16, device=DEV)
    table = (n_pages - 1 - torch.arange(24, device=DEV, dtype=torch.int32)).view(2, 12)
    lens = [2500, 300]
    c = kvd.LatentCache(kvd.BF16, 2, n_pages, page, 12, tensors={
        "rows": rows, "page_table": table, "seq_lens": torch.tensor(lens, dtype=torch.int32, device=DEV)})
    c.len = 2500
    rows[-24:].copy_(torch.randn(24, page, rank + P, generator=_gen(1), device=DEV))
    lat, k = _q(2, 1, rank, torch.bfloat16, 2)[:, 0], _q(2, 1, P, torch.bfloat16, 3)[:, 0]
    kvd.latent_append(c, lat, k, _starts([1, 1]))
    for b, n in enumerate(lens):
        assert torch.equal(rows[int(table[b, (n - 1) // page]), (n - 1) % page], torch.cat([lat[b], k[b]]))
    q = _q(2, 16, 576, torch.bfloat16, 4)
    _, lse = _check(c, q, [1, 1])
    mass = torch.zeros(2, 1, 2500, device=DEV)
    kvd.paged_mass(c, q, lse, _starts([1, 1]), 1, 0.07, mass)
    want = LR.attn(c, q, [0, 1, 2], lens, 0.07, 0, 1.0, torch.zeros_like(mass))
    LR.assert_close(mass, want["mass"])
    to = (torch.arange(4, device=DEV, dtype=torch.int32) + n_pages - 30).view(2, 2)
    kept = torch.empty(2, 1, 400, dtype=torch.int32, device=DEV)
    new = torch.empty(2, dtype=torch.int32, device=DEV)
    kvd.paged_evict(c, mass, 400, to, kept, new)
    assert new.tolist() == [400, 300] and c.device_status() == 0
    ids = kept[0, 0].long()
    got = rows[to[0].long()].flatten(0, 1)[:400]
    assert torch.equal(got, rows[table[0].long()].flatten(0, 1)[ids])
