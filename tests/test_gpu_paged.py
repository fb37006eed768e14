"""kvd_paged_append and kvd_paged_attn against 64-bit references (bounds in paged_ref.py)."""
import math

import pytest
import torch

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


def _cache(dtype, lens, Hkv, D, page, seed, fill=True, spare=1):
    """A cache of scattered pages that hold data in every row (stale ones too)."""
    B = len(lens)
    cols = max(1, max((n + page - 1) // page for n in lens)) + spare
    c = kvd.PagedKVCache(dtype, B, B * cols, Hkv, page, cols, head_dim=D)
    c.page_table.copy_(R.scattered_tables(B, cols, seed, DEV))
    c.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
    c.len = max(lens)
    g = _gen(seed)
    for n in "kv":
        p = c.t[n]
        if dtype == kvd.INT8:
            p.copy_(torch.randint(-127, 128, p.shape, generator=g, device=DEV))
            c.t[n + "_scale"].copy_(torch.rand(p.shape[:3], generator=g, device=DEV) * 0.02 + 0.001)
        else:
            p.copy_(torch.randn(p.shape, generator=g, device=DEV))
    return c


def _attend(c, q, new, window=0, scale=None, out=None, ws=None, max_new=None):
    scale = scale or q.shape[2] ** -0.5
    out = torch.full_like(q, math.nan) if out is None else out
    T = q.shape[0]
    max_new = max_new or max(new)
    ws = kvd.make_paged_workspace(c, q.shape[1], T, max_new) if ws is None else ws
    kvd.paged_attn(c, q, _starts(new), max_new, scale, out, ws, window=window)
    return out


def _check_attn(c, q, new, window=0, scale=None, **kw):
    scale = scale or q.shape[2] ** -0.5
    out = _attend(c, q, new, window, scale, **kw)
    want, tol = R.attn_ref(c, q, _starts(new).tolist(), c.seq_lens.tolist(), scale, window)
    n = sum(new)
    R.assert_within(out[:n], want[:n], tol[:n])
    assert c.device_status() == 0
    return out


def _q(T, H, D, x, seed, scale=1.0):
    return (torch.randn(T, H, D, generator=_gen(seed), device=DEV) * scale).to(x)


# ----------------------------------------------------------------- append ---

@pytest.mark.parametrize("dtype", [kvd.F16, kvd.BF16, kvd.INT8])
@pytest.mark.parametrize("x", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page,D,inter,norm", [(16, 128, False, True), (48, 64, True, False),
                                               (64, 128, True, True), (256, 64, False, False)])
def test_append(dtype, x, page, D, inter, norm):
    Hkv, H = 3, 6
    new, lens = [5, 0, 1, 130, 17], [5, 40, 65, 200, 400]
    T = sum(new) + 3                                  # three padding rows behind the last sequence
    c = _cache(dtype, lens, Hkv, D, page, page + D)
    before = {n: c.t[n].clone() for n in c.t}
    g = _gen(3)
    x_all = (torch.randn(T, H + 2 * Hkv, D, generator=g, device=DEV) * 3).to(x)
    q, k, v = x_all[:, :H], x_all[:, H:H + Hkv], x_all[:, H + Hkv:]
    w = [torch.rand(D, generator=g, device=DEV) + 0.5 for _ in range(2)] if norm else [None, None]
    q_out = torch.full((T, H, D), 7.0, device=DEV, dtype=x)
    rope = kvd.rope_table(D, interleaved=inter, scaling="yarn", factor=4, orig_len=4096)
    kvd.paged_append(c, k, v, _starts(new), rope=rope, k_weight=w[1], q=q, q_out=q_out, q_weight=w[0])
    assert c.device_status() == 0
    f, m = R.freqs(D, 10000.0, "yarn", 4, 4096)
    t = 0
    touched = torch.zeros(c.n_pages, page, dtype=torch.bool, device=DEV)
    for b, n in enumerate(new):
        for i in range(n):
            p = lens[b] - n + i
            pos = torch.tensor([p], device=DEV)
            at = int(c.page_table[b, p // page]), p % page
            touched[at] = True
            y, err = R.turned(q[t:t + 1], pos, f, m, inter, w[0])
            R.assert_within(q_out[t:t + 1], y, R.rounding(y, err, x), "q")
            yk, ek = R.turned(k[t:t + 1], pos, f, m, inter, w[1])
            for name, (y, err) in (("k", (yk[0], ek[0])), ("v", (v[t].double(), torch.zeros_like(yk[0])))):
                got = c.t[name][at[0], :, at[1]]
                if dtype == kvd.INT8:
                    s = c.t[name + "_scale"][at[0], :, at[1]].double()
                    a = y.abs().amax(-1)
                    assert torch.all((s - a / 127).abs() <= err.amax(-1) / 127 + a / 127 * 2.0 ** -23)
                    # half a code, and what the row and its scale are off by
                    assert torch.all((got.double() * s[:, None] - y).abs() <=
                                     s[:, None] * (0.5 + 2.0 ** -14) + 2 * err)
                    assert int(got.abs().max()) <= 127
                else:
                    R.assert_within(got, y, R.rounding(y, err, X[dtype]), name)
            t += 1
    assert torch.all(q_out[t:] == 7.0)                # padding rows left as they were
    for n in ("k", "v", "k_scale", "v_scale"):
        if n in c.t:
            keep = ~touched[:, None, :].expand(c.n_pages, Hkv, page)
            assert torch.equal(c.t[n][keep], before[n][keep]), n


@pytest.mark.parametrize("dtype", [kvd.F16, kvd.INT8])
@pytest.mark.parametrize("x", [torch.float16, torch.float32])
def test_append_without_rotation_stores_what_kv_append_stores(dtype, x):
    B, n, Hkv = 2, 77, 4
    k = (torch.randn(B, n, Hkv, 128, generator=_gen(1), device=DEV) * 4).to(x)
    v = torch.randn(B, n, Hkv, 128, generator=_gen(2), device=DEV).to(x)
    k[0, 3, 1] = 0                                     # a row whose scale is zero
    old = kvd.KVCache(dtype, B, Hkv, 128)
    (kvd.kv_append if x == torch.float16 else kvd.kv_append_f32)(old, k, v)
    new = kvd.KVCache(dtype, B, Hkv, 128)
    new.len = n
    over = kvd.PagedKVCache.over(new)
    kvd.paged_append(over, k.flatten(0, 1), v.flatten(0, 1), _starts([n, n]))
    for t in ("k", "v", "k_scale", "v_scale"):
        if t in old.t:
            assert torch.equal(old.t[t][:, :, :n], new.t[t][:, :, :n]), t


def test_append_checks_what_the_device_holds():
    """Bad pages and lengths are reported and skipped; the other sequences are served."""
    def fresh():
        c = _cache(kvd.F16, [20, 20, 20], 2, 64, 16, 5)
        k = _q(12, 2, 64, torch.float16, 6)
        return c, k, {n: c.t[n].clone() for n in ("k", "v")}

    for col, bad in ((1, -1), (1, 10 ** 6)):
        c, k, before = fresh()
        c.page_table[1, col] = bad
        kvd.paged_append(c, k, k, _starts([4, 4, 4]))
        assert c.device_status() == 1
        changed = (c.k != before["k"]).any(-1).any(1)          # [pages, page]
        assert int(changed.sum()) == 8
        for b in (0, 2):
            assert changed[int(c.page_table[b, 1]), :4].all()
    c, k, before = fresh()
    c.seq_lens[1] = 2                                           # four new tokens in a length of two
    kvd.paged_append(c, k, k, _starts([4, 4, 4]))
    assert c.device_status() == 1
    changed = (c.k != before["k"]).any(-1).any(1)
    assert int(changed.sum()) == 10 and changed[int(c.page_table[1, 0]), :2].all()
    c, k, before = fresh()
    c.seq_lens[1] = 21                                          # above len: moved to it
    kvd.paged_append(c, k, k, _starts([4, 4, 4]))
    assert c.device_status() == 1
    assert int((c.k != before["k"]).any(-1).any(1).sum()) == 12
    c, k, before = fresh()
    kvd.paged_append(c, k, k, torch.tensor([0, 8, 4, 12], dtype=torch.int32, device=DEV))
    assert c.device_status() == 1


def test_starts_outside_the_tokens_are_moved_into_them():
    """A first start below 0 and a last one above n_tokens: reported, and both calls take the same rows."""
    c = _cache(kvd.F16, [20, 20, 20], 2, 64, 16, 5)
    k = _q(12, 2, 64, torch.float16, 6)
    before = c.k.clone()
    starts = torch.tensor([-2, 4, 8, 15], dtype=torch.int32, device=DEV)
    kvd.paged_append(c, k, k, starts)
    assert c.device_status() == 1
    for b in range(3):
        page = int(c.page_table[b, 1])                          # positions 16 .. 19
        assert torch.equal(c.k[page, :, :4].transpose(0, 1), k[4 * b:4 * b + 4])
    assert int((c.k != before).any(-1).any(1).sum()) == 12
    out = torch.full_like(k, math.nan)
    kvd.paged_attn(c, k, starts, 4, 0.125, out, kvd.make_paged_workspace(c, 2, 12, 4))
    assert c.device_status() == 1
    want, tol = R.attn_ref(c, k, [0, 4, 8, 12], [20, 20, 20], 0.125)
    R.assert_within(out, want, tol)


def test_append_a_large_batch_finds_every_token():
    B = 1500
    lens = [1 + b % 37 for b in range(B)]
    new = [b % 3 if b % 3 <= lens[b] else 1 for b in range(B)]
    c = _cache(kvd.BF16, lens, 1, 64, 16, 8)
    k = _q(sum(new), 1, 64, torch.bfloat16, 9)
    kvd.paged_append(c, k, k, _starts(new))
    assert c.device_status() == 0
    t, page, slot = [], [], []
    table = c.page_table.tolist()
    for b, n in enumerate(new):
        for p in range(lens[b] - n, lens[b]):
            page.append(table[b][p // 16])
            slot.append(p % 16)
    assert torch.equal(c.k[torch.tensor(page), :, torch.tensor(slot)], k)


# -------------------------------------------------------------- attention ---

LENS = [1, 63, 64, 65, 127, 128, 129, 300, 1000]


@pytest.mark.parametrize("dtype,x", [(kvd.F16, torch.float16), (kvd.BF16, torch.bfloat16),
                                     (kvd.INT8, torch.float16), (kvd.INT8, torch.bfloat16)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 48, 64, 256])
@pytest.mark.parametrize("G", [1, 4, 7])
def test_single_tokens(dtype, x, D, page, G):
    Hkv = 2
    c = _cache(dtype, LENS, Hkv, D, page, page + G)
    _check_attn(c, _q(len(LENS), Hkv * G, D, x, G), [1] * len(LENS))


@pytest.mark.parametrize("dtype,x", [(kvd.F16, torch.float16), (kvd.BF16, torch.bfloat16),
                                     (kvd.INT8, torch.float16), (kvd.INT8, torch.bfloat16)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 80, 128])
@pytest.mark.parametrize("G", [1, 3, 8])
@pytest.mark.parametrize("window", [0, 1, 100])
def test_ragged_chunks(dtype, x, D, page, G, window):
    Hkv = 2
    new = [1, 0, 200, 64, 5, 129, 17]
    lens = [300, 10, 200, 65, 1000, 130, 17]
    c = _cache(dtype, lens, Hkv, D, page, page + G + window)
    _check_attn(c, _q(sum(new), Hkv * G, D, x, G), new, window)


@pytest.mark.parametrize("dtype,x", [(kvd.F16, torch.float16), (kvd.BF16, torch.bfloat16),
                                     (kvd.INT8, torch.float16)])
@pytest.mark.parametrize("new,L,H,Hkv,D", [(1, 20011, 8, 8, 128), (1, 70000, 16, 1, 128), (3, 33333, 32, 8, 64),
                                           (100, 9000, 4, 1, 128), (700, 5000, 8, 2, 128),
                                           (1500, 1500, 4, 4, 64), (16, 16, 16, 1, 128)])
def test_long_and_split(dtype, x, new, L, H, Hkv, D):
    c = _cache(dtype, [L], Hkv, D, 64, L)
    _check_attn(c, _q(new, H, D, x, L, scale=2.0), [new])


@pytest.mark.parametrize("window", [1, 2, 64, 127, 128, 129, 5000])
@pytest.mark.parametrize("new", [1, 9, 300])
def test_windows(window, new):
    c = _cache(kvd.F16, [4100, 350], 2, 128, 16, window)
    _check_attn(c, _q(2 * new, 8, 128, torch.float16, window), [new, new], window)


@pytest.mark.parametrize("dtype", [kvd.F16, kvd.BF16, kvd.INT8])
@pytest.mark.parametrize("new,lens,window", [([1, 1], [70, 1], 0), ([40, 130], [200, 130], 0),
                                             ([1, 60], [500, 700], 100), ([300, 2], [1000, 131], 50)])
@pytest.mark.parametrize("page", [16, 128, 256])
def test_dead_rows_may_hold_anything(dtype, new, lens, window, page):
    """NaN and infinities in rows no token may see: behind the length, and before the window."""
    c = _cache(dtype, lens, 2, 128, page, 77)
    x = X.get(dtype, torch.bfloat16)
    q = _q(sum(new), 8, 128, x, 5)
    clean = _check_attn(c, q, new, window)
    for b, (n, L) in enumerate(zip(new, lens)):
        first = max(0, L - n - window + 1) if window else 0
        for p in range(c.max_pages * page):
            if p >= L or p < first:
                pg, off = int(c.page_table[b, p // page]), p % page
                bad = (math.nan, math.inf, -math.inf)[p % 3]
                for n_ in ("k_scale", "v_scale") if dtype == kvd.INT8 else ("k", "v"):
                    c.t[n_][pg, :, off] = bad
        for j in range(c.max_pages):                   # pages nothing needs are not even looked at
            if j * page >= L or (j + 1) * page <= first:
                c.page_table[b, j] = -12345
    assert torch.equal(_attend(c, q, new, window), clean)
    assert c.device_status() == 0


def test_rows_that_see_nothing_and_padding():
    """Empty sequences, padding rows behind the last one, and new tokens before position 0."""
    c = _cache(kvd.F16, [5, 0, 3], 1, 64, 16, 3)
    q = _q(20, 4, 64, torch.float16, 4)
    out = torch.full_like(q, 9.0)
    _check_attn(c, q, [2, 0, 1], out=out)
    assert torch.all(out[3:] == 9.0)
    c.seq_lens[2] = 1                                  # three new tokens in a length of one
    out = _attend(c, q, [2, 0, 3], out=torch.full_like(q, 9.0))
    assert c.device_status() == 1
    assert not out[2:4].any() and bool(out[4].any()) and torch.all(out[5:] == 9.0)


def test_max_new_too_small_is_reported():
    c = _cache(kvd.F16, [50, 400], 1, 64, 16, 3)
    q = _q(310, 4, 64, torch.float16, 4)
    out = torch.full_like(q, 9.0)
    ws = kvd.make_paged_workspace(c, 4, 310, 300)
    kvd.paged_attn(c, q, _starts([10, 300]), 20, 0.125, out, ws)
    assert c.device_status() == 1
    want, tol = R.attn_ref(c, q, [0, 10, 310], [50, 400], 0.125)
    R.assert_within(out[:10], want[:10], tol[:10])
    R.assert_within(out[10:30], want[10:30], tol[10:30])
    assert torch.all(out[30:] == 9.0)


def test_bad_pages_are_left_out():
    c = _cache(kvd.F16, [100, 100], 1, 64, 16, 3)
    q = _q(2, 4, 64, torch.float16, 4)
    good = _attend(c, q, [1, 1])
    c.page_table[0, 2] = -1
    c.page_table[0, 4] = c.n_pages
    out = _attend(c, q, [1, 1])
    assert c.device_status() == 1
    assert torch.equal(out[1], good[1]) and bool(torch.isfinite(out).all())
    # the same keys and values gathered without the two pages
    rows = [i for i in range(100) if i // 16 not in (2, 4)]
    k = torch.stack([c.k[int(c.page_table[0, i // 16]), 0, i % 16] for i in rows]).double()
    v = torch.stack([c.v[int(c.page_table[0, i // 16]), 0, i % 16] for i in rows]).double()
    for h in range(4):
        p = torch.softmax(k @ q[0, h].double() * 64 ** -0.5, 0)
        assert (out[0, h].double() - p @ v).norm() <= 2e-3 * (p @ v).norm()


@pytest.mark.parametrize("dtype", [kvd.F16, kvd.INT8])
def test_growing_logits_and_tiny_values(dtype):
    """The running maximum rises through the whole cache; values near the type's smallest."""
    L, D = 3000, 128
    c = _cache(dtype, [L, L], 1, D, 64, 12)
    q = _q(2, 8, D, torch.float16, 13)
    unit = q[0, 0].float() / q[0, 0].float().norm()
    for p in range(L):
        pg, off = int(c.page_table[0, p // 64]), p % 64
        row = unit * (p / 40.0)
        if dtype == kvd.INT8:
            s = row.abs().max() / 127
            c.k[pg, 0, off] = (row / max(float(s), 1e-9)).round().to(torch.int8)
            c.k_scale[pg, 0, off] = s
            c.v_scale[pg, 0, off] = 1e-9 * (1 + p % 7) * (1000.0 if p % 500 == 0 else 1.0)
        else:
            c.k[pg, 0, off] = row.half()
    _check_attn(c, q, [1, 1])
    if dtype == kvd.F16:
        c.v.mul_(1e-3)
        _check_attn(c, q, [1, 1])


@pytest.mark.parametrize("dtype", [kvd.F16, kvd.BF16, kvd.INT8])
@pytest.mark.parametrize("new,L,G,window", [(20, 140, 1, 8), (7, 1030, 4, 5), (30, 1300, 1, 100), (60, 170, 2, 8)])
def test_rows_whose_first_keys_come_in_a_later_tile(dtype, new, L, G, window):
    """A window hides the first tile from the last tokens, and their logits are far below zero."""
    D = 128
    x = X.get(dtype, torch.float16)
    c = _cache(dtype, [L], 1, D, 64, 21)
    k = torch.randn(c.k.shape, generator=_gen(22), device=DEV) * 0.3 + 2.0
    if dtype == kvd.INT8:
        c.k_scale.copy_(k.abs().amax(-1) / 127)
        c.k.copy_((k / c.k_scale[..., None]).round())
    else:
        c.k.copy_(k)
    q = (torch.randn(new, G, D, generator=_gen(23), device=DEV) * 0.3 - 2.0).to(x)
    _check_attn(c, q, [new], window)


@pytest.mark.parametrize("dtype", [kvd.F16, kvd.INT8])
@pytest.mark.parametrize("new", [1, 30, 300])
def test_a_window_longer_than_any_sequence(dtype, new):
    c = _cache(dtype, [1000, 700], 2, 128, 64, 24)
    q = _q(2 * new, 2, 128, torch.float16, 25)
    plain = _attend(c, q, [new, new])
    for window in (1000, 1001, 2 ** 30, 2 ** 31 - 1):
        assert torch.equal(_attend(c, q, [new, new], window), plain)


@pytest.mark.parametrize("dtype,x", [(kvd.F16, torch.float16), (kvd.BF16, torch.bfloat16),
                                     (kvd.INT8, torch.float16), (kvd.INT8, torch.bfloat16)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,new", [(4, [9, 30, 1, 0]), (16, [3, 8, 8, 1]), (1, [33, 128, 2, 100])])
@pytest.mark.parametrize("window", [0, 70])
def test_33_to_128_rows(dtype, x, D, G, new, window):
    lens = [5000, 300, 77, 129]
    c = _cache(dtype, lens, 2, D, 48, D + G + window)
    _check_attn(c, _q(sum(new), 2 * G, D, x, G, scale=1.5), new, window)


@pytest.mark.parametrize("dtype", [kvd.F16, kvd.INT8])
@pytest.mark.parametrize("B,every,longest", [(1500, 3, 2), (700, 50, 40), (400, 7, 20), (45, 4, 90)])
def test_large_batches(dtype, B, every, longest):
    """More sequences than a block has threads, most of one token, some with none, a few with more."""
    lens = [1 + b * 37 % 301 for b in range(B)]
    new = [min(longest if b % every == 0 else b % every % 2, lens[b]) for b in range(B)]
    c = _cache(dtype, lens, 1, 64, 32, B)
    _check_attn(c, _q(sum(new), 4, 64, torch.float16, B), new, max_new=longest)


@pytest.mark.parametrize("dtype", [kvd.F16, kvd.INT8])
def test_one_workspace_for_calls_of_every_length(dtype):
    """Made for the longest, used by chunks and single tokens in turn, and by two graphs of them."""
    H, D = 8, 128
    c = _cache(dtype, [4000, 900], 2, D, 64, 26)
    ws = kvd.make_paged_workspace(c, H, 600, 300)
    sizes = [300, 1, 20, 8, 300, 2, 1]
    q = {n: _q(2 * n, H, D, torch.float16, n) for n in sizes}
    want = {n: _attend(c, q[n], [n, n]) for n in sizes}
    for n in sizes:
        assert torch.equal(_attend(c, q[n], [n, n], ws=ws), want[n])
    graphs, outs = {}, {n: torch.full_like(q[n], math.nan) for n in (300, 1)}
    starts = {n: _starts([n, n]) for n in (300, 1)}
    for n in (300, 1):
        graphs[n] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[n]):
            kvd.paged_attn(c, q[n], starts[n], n, D ** -0.5, outs[n], ws)
    for n in (300, 1, 1, 300, 1):
        outs[n].fill_(math.nan)
        graphs[n].replay()
        assert torch.equal(outs[n], want[n])
    assert c.device_status() == 0


def test_strided_queries_and_outputs():
    c = _cache(kvd.BF16, [90, 33], 2, 128, 32, 14)
    wide = torch.randn(12, 14, 128, device=DEV).bfloat16()
    q = wide[:, 2:10]
    big = torch.zeros(12, 20, 128, device=DEV, dtype=torch.bfloat16)
    _check_attn(c, q, [7, 5], out=big[:, 8:16])
    assert not big[:, :8].any() and not big[:, 16:].any()


@pytest.mark.parametrize("dtype", [kvd.F16, kvd.INT8])
def test_a_contiguous_cache_as_pages(dtype):
    """Chunk attention over a KVCache, next to the decode call on the same cache."""
    B, L, Hkv, H = 2, 777, 2, 8
    cache = kvd.KVCache(dtype, B, Hkv, 1024)
    k = torch.randn(B, L, Hkv, 128, generator=_gen(1), device=DEV).half()
    v = torch.randn(B, L, Hkv, 128, generator=_gen(2), device=DEV).half()
    kvd.kv_append(cache, k, v)
    p = kvd.PagedKVCache.over(cache)
    q = _q(2 * 50, H, 128, torch.float16, 3)
    out = _check_attn(p, q, [50, 50])
    last = q.view(B, 50, H, 128)[:, -1].float().contiguous()
    dec = torch.empty(B, H, 128, device=DEV)
    kvd.decode_attn_dense(cache, last, 128 ** -0.5, dec, kvd.make_workspace(cache, H))
    got = out.view(B, 50, H, 128)[:, -1].float()
    # int8: the decode call rounds the query to 8 bits too
    assert (got - dec).norm() <= (2e-3 if dtype == kvd.F16 else 2e-2) * dec.norm()


@pytest.mark.parametrize("dtype,x", [(kvd.F16, torch.float16), (kvd.BF16, torch.bfloat16),
                                     (kvd.INT8, torch.bfloat16)])
def test_prefill_then_decode_steps(dtype, x):
    """A prompt in two chunks, then single tokens: each step appends (norm, rotation) and attends."""
    H, Hkv, D, page, total = 8, 2, 128, 16, 300
    c = kvd.PagedKVCache(dtype, 1, 40, Hkv, page, 20, head_dim=D)
    c.page_table.copy_(torch.randperm(40, device=DEV)[:20].view(1, -1))
    qkv = _q(total, H + 2 * Hkv, D, x, 31)
    w = [torch.rand(D, generator=_gen(i), device=DEV) + 0.5 for i in (1, 2)]
    rope = kvd.rope_table(64, interleaved=True)
    ws = kvd.make_paged_workspace(c, H, 200, 200)
    done, outs, qs = 0, [], []
    for n in [200, 93] + [1] * 7:
        x_ = qkv[done:done + n]
        done += n
        c.seq_lens.fill_(done)
        c.len = done
        q, out = torch.empty(n, H, D, dtype=x, device=DEV), torch.empty(n, H, D, dtype=x, device=DEV)
        kvd.paged_append(c, x_[:, H:H + Hkv], x_[:, H + Hkv:], _starts([n]), rope=rope, k_weight=w[1],
                         q=x_[:, :H], q_out=q, q_weight=w[0])
        kvd.paged_attn(c, q, _starts([n]), n, D ** -0.5, out, ws)
        outs.append(out)
        qs.append(q)
    assert c.device_status() == 0
    q = torch.cat(qs)
    y, err = R.turned(qkv[:, :H], torch.arange(total, device=DEV), *R.freqs(64), True, w[0])
    R.assert_within(q, y, R.rounding(y, err, x))
    want, tol = R.attn_ref(c, q, [0, total], [total], D ** -0.5)
    R.assert_within(torch.cat(outs), want, tol)


@pytest.mark.parametrize("dtype", [kvd.F16, kvd.INT8])
def test_same_bits_twice_and_in_a_replayed_graph(dtype):
    """A captured step replayed after its device-side lengths, tables and inputs changed."""
    B, H, Hkv, D, page = 3, 8, 2, 128, 16
    c = _cache(dtype, [900, 40, 333], Hkv, D, page, 41, spare=8)
    c.len = 1000
    new = [1, 1, 1]
    x = torch.float16
    qkv = _q(B, H + 2 * Hkv, D, x, 42)
    q, out = torch.empty(B, H, D, dtype=x, device=DEV), torch.empty(B, H, D, dtype=x, device=DEV)
    rope, starts = kvd.rope_table(128), _starts(new)
    ws = kvd.make_paged_workspace(c, H, B, 1)

    def step():
        kvd.paged_append(c, qkv[:, H:H + Hkv], qkv[:, H + Hkv:], starts, rope=rope, q=qkv[:, :H], q_out=q)
        kvd.paged_attn(c, q, starts, 1, D ** -0.5, out, ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    first = out.clone()
    step()
    assert torch.equal(out, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        c.seq_lens.add_(torch.tensor([1, 17, 0], dtype=torch.int32, device=DEV))
        c.page_table.copy_(c.page_table.flip(0).clone())
        qkv.copy_(_q(B, H + 2 * Hkv, D, x, 50 + i))
        out.fill_(math.nan)
        graph.replay()
        replayed = out.clone()
        want, tol = R.attn_ref(c, q, starts.tolist(), c.seq_lens.tolist(), D ** -0.5)
        R.assert_within(replayed, want, tol)
        step()
        assert torch.equal(out, replayed)
    assert c.device_status() == 0


def test_two_streams_with_a_workspace_each():
    c = [_cache(kvd.F16, [2500], 2, 128, 64, 60 + i) for i in range(2)]
    q = [_q(130, 8, 128, torch.float16, 70 + i) for i in range(2)]
    want = [_attend(a, b, [130]) for a, b in zip(c, q)]
    ws = [kvd.make_paged_workspace(a, 8, 130, 130) for a in c]
    outs = [torch.full_like(b, math.nan) for b in q]
    starts = _starts([130])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, s in enumerate(streams):
            kvd.paged_attn(c[i], q[i], starts, 130, 128 ** -0.5, outs[i], ws[i], stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_offsets_beyond_31_bits():
    """Pages whose byte and element offsets pass 2^31 and 2^32."""
    page, Hkv, D = 64, 8, 128
    n_pages = 70000                                     # 36.7 G rows' channels: 9.2 GB a side
    c = kvd.PagedKVCache(kvd.F16, 2, n_pages, Hkv, page, 4, head_dim=D)
    ids = torch.tensor([[69999, 33000, 65537, 0], [1, 40000, 32768, 69998]], dtype=torch.int32)
    c.page_table.copy_(ids)
    lens = [200, 250]
    c.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
    c.len = 250
    k = _q(450, Hkv, D, torch.float16, 3)
    v = _q(450, Hkv, D, torch.float16, 4)
    kvd.paged_append(c, k, v, _starts(lens))
    assert torch.equal(torch.cat([R.rows_of(c.k, c.page_table[b], lens[b], 7) for b in range(2)]), k[:, 7])
    q = _q(450, Hkv, D, torch.float16, 5)
    _check_attn(c, q, lens)


def test_perf_cases_agree():
    """The plain forms and the calls of perf/operators.py, on small drawn cases."""
    import importlib.util
    import os
    import random
    at = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "operators.py")
    spec = importlib.util.spec_from_file_location("perf_operators", at)
    M = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(M)
    rng = random.Random(12)
    done = 0
    while done < 12:
        case = M.draw(rng)
        if M.work(case)["flops"] > 2e10 or M.work(case)["bytes"] > 5e7:
            continue
        done += 1
        got = []
        for own in (False, True):
            M.own = own
            r = M.run(M.prepare(case, 5))
            got.append([t.double().clone() for t in (r if isinstance(r, tuple) else (r,))])
        for a, b in zip(*got):
            assert (a - b).norm() <= 1e-2 * a.norm(), case
