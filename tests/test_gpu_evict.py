"""Statistics of the paged attention, accumulated weights, and eviction, against 64-bit references
(bounds in latent_ref.py); the eviction is exact."""
import math

import pytest
import torch

import latent_ref as LR
import long_context_decode_kv_gb300 as kvd
import paged_ref as R
from test_gpu_latent import _cache as _latent
from test_gpu_latent import _attend as _latent_attend
from test_gpu_paged import _cache as _paged
from test_gpu_paged import _gen, _q, _starts

pytestmark = pytest.mark.gpu
DEV = "cuda"
X = {kvd.F16: torch.float16, kvd.BF16: torch.bfloat16, kvd.INT8: torch.float16}


def _attend(c, q, new, window=0, scale=0.1):
    if isinstance(c, kvd.LatentCache):
        return _latent_attend(c, q, new, window, scale)
    out, lse = torch.full_like(q, math.nan), torch.full(q.shape[:2], math.nan, device=DEV)
    ws = kvd.make_paged_workspace(c, q.shape[1], q.shape[0], max(new))
    kvd.paged_attn(c, q, _starts(new), max(new), scale, out, ws, window=window, lse=lse)
    return out, lse


def _check(c, q, new, window=0, scale=0.1, decay=1.0, spare=5):
    heads = LR.heads_of(c)
    mass = torch.rand(c.batch, heads, c.len + spare, generator=_gen(11), device=DEV) * 0.1
    _, lse = _attend(c, q, new, window, scale)
    want = LR.attn(c, q, _starts(new).tolist(), c.seq_lens.tolist(), scale, window, decay, mass)
    LR.assert_close(lse, want["lse"], "lse")
    out = torch.full_like(mass, 7.0)
    kvd.paged_mass(c, q, lse, _starts(new), max(new), scale, mass, out=out, decay=decay, window=window)
    assert c.device_status() == 0
    LR.assert_close(out, want["mass"], "mass")
    assert torch.all(out[want["mass"][0].isnan()] == 7.0)      # behind a sequence's length
    again = mass.clone()
    kvd.paged_mass(c, q, lse, _starts(new), max(new), scale, again, decay=decay, window=window)
    some = ~want["mass"][0].isnan()
    assert torch.equal(again[some], out[some])                  # in place, and the same bits
    assert torch.equal(again[~some], mass[~some])
    return out


# ------------------------------------------------------------- statistics ---

@pytest.mark.parametrize("dtype", [kvd.F16, kvd.BF16, kvd.INT8])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv,new,lens", [
    (8, 2, [1, 1, 1], [1, 300, 20000]), (32, 4, [3, 1, 4], [3, 129, 900]),
    (8, 2, [20, 0, 9], [20, 50, 5000]), (8, 8, [200, 1, 129], [1000, 128, 129])])
def test_paged_lse(dtype, D, H, Hkv, new, lens):
    """Single tokens, 32 rows, row tiles alone and in pairs, items whole and cut; the output stays."""
    c = _paged(dtype, lens, Hkv, D, 64, D)
    q = _q(sum(new) + 1, H, D, X[dtype], 5)
    for window in (0, 70):
        out, lse = _attend(c, q, new, window)
        want = LR.attn(c, q, _starts(new).tolist(), lens, 0.1, window)
        LR.assert_close(lse, want["lse"])
        assert lse[sum(new):].isnan().all()
        plain = torch.full_like(q, math.nan)
        ws = kvd.make_paged_workspace(c, H, q.shape[0], max(new))
        kvd.paged_attn(c, q, _starts(new), max(new), 0.1, plain, ws, window=window)
        assert torch.equal(plain[:sum(new)], out[:sum(new)])


def test_paged_lse_of_rows_without_keys():
    for new, n in (([5], 5), ([60], 60)):
        c = _paged(kvd.F16, [3], 2, 64, 16, 2)
        c2 = _q(n, 8, 64, torch.float16, 3)
        out, lse = _attend(c, c2, new)
        assert c.device_status() == 1
        assert torch.all(lse[:n - 3] == -math.inf) and torch.all(out[:n - 3] == 0)
        assert lse[n - 3:].isfinite().all()


# ----------------------------------------------------- accumulated weights ---

@pytest.mark.parametrize("dtype", [kvd.F16, kvd.BF16, kvd.INT8])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 48), (128, 64), (64, 128)])
@pytest.mark.parametrize("H,Hkv", [(4, 4), (7, 1), (32, 8), (16, 1)])
def test_mass_of_single_tokens(dtype, D, page, H, Hkv):
    lens = [1, 127, 128, 129, 700, 3]
    c = _paged(dtype, lens, Hkv, D, page, D + page)
    _check(c, _q(6, H, D, X[dtype], 5), [1] * 6, decay=0.9)


@pytest.mark.parametrize("dtype", [kvd.F16, kvd.BF16, kvd.INT8])
@pytest.mark.parametrize("window", [0, 1, 60, 128, 333])
def test_mass_of_ragged_batches(dtype, window):
    new, lens = [1, 300, 0, 20, 7, 129], [500, 300, 260, 1000, 7, 400]
    c = _paged(dtype, lens, 2, 128, 32, 4)
    _check(c, _q(sum(new) + 2, 10, 128, X[dtype], 5), new, window=window)


def test_mass_with_bf16_queries_over_int8():
    c = _paged(kvd.INT8, [200, 900], 2, 64, 16, 4)
    _check(c, _q(45, 8, 64, torch.bfloat16, 5), [5, 40], decay=0.5)


@pytest.mark.parametrize("dtype", [kvd.F16, kvd.BF16])
@pytest.mark.parametrize("rank,P,H,new", [(512, 64, 128, [1, 1, 1]), (512, 64, 16, [1, 20, 0]),
                                          (256, 32, 40, [9, 1, 70]), (128, 16, 130, [1, 3, 2]),
                                          (384, 48, 7, [30, 1, 1])])
def test_mass_of_latent_rows(dtype, rank, P, H, new):
    c = _latent(dtype, [100, 900, 260], 16, rank, rank, P)
    _check(c, _q(sum(new), H, rank + P, X[dtype], 5), new, scale=0.06, window=0 if H != 40 else 50)


def test_mass_of_a_step_sums_to_the_rows():
    """The weights of a row add up to 1: of a head, to its rows."""
    c = _paged(kvd.BF16, [5000, 77], 2, 128, 64, 4)
    q = _q(3, 8, 128, torch.bfloat16, 5)
    _, lse = _attend(c, q, [2, 1])
    out = torch.zeros(2, 2, 5000, device=DEV)
    kvd.paged_mass(c, q, lse, _starts([2, 1]), 2, 0.1, None, out=out, decay=0.0)
    rows = torch.tensor([8.0, 4.0], device=DEV)[:, None].expand(2, 2)
    _, tol = LR.attn(c, q, [0, 2, 3], [5000, 77], 0.1, 0, 0.0, torch.zeros_like(out))["mass"]
    assert torch.all((out.double().sum(-1) - rows).abs() <= tol.sum(-1))


def test_mass_decay_alone():
    """No new tokens at all, and a sequence without any beside one with some."""
    c = _paged(kvd.F16, [100, 60], 2, 64, 16, 4)
    mass = torch.rand(2, 2, 128, generator=_gen(3), device=DEV)
    q = torch.empty(0, 4, 64, dtype=torch.float16, device=DEV)
    out = torch.full_like(mass, 7.0)
    kvd.paged_mass(c, q, torch.empty(0, 4, device=DEV), _starts([0, 0]), 0, 0.1, mass, out=out, decay=0.25)
    for b, n in enumerate((100, 60)):
        assert torch.equal(out[b, :, :n], mass[b, :, :n] * 0.25) and torch.all(out[b, :, n:] == 7.0)
    assert c.device_status() == 0


def test_mass_leaves_out_what_no_row_sees():
    """Rows without a key, bad pages, stale rows, another sequence's NaN queries."""
    c = _paged(kvd.F16, [3, 200, 64], 1, 64, 16, 2)
    q = _q(5 + 4 + 8, 4, 64, torch.float16, 3)
    new = [5, 4, 8]
    _, lse = _attend(c, q, new)
    assert c.device_status() == 1 and torch.all(lse[:2] == -math.inf)
    c.t["status"].zero_()
    zero = torch.zeros(3, 1, 256, device=DEV)
    want = torch.zeros_like(zero)
    kvd.paged_mass(c, q, lse, _starts(new), 8, 0.1, zero, out=want)
    c.t["status"].zero_()
    # three rows of four heads; logits off by 2 * 64 steps of 2^-23 of sums below 16
    assert (want[0, 0, :3].double().sum() - 12).abs() < 12 * 4 * 64 * 2.0 ** -23 * 16
    used = torch.zeros(c.n_pages, 16, dtype=torch.bool, device=DEV)
    for b, l in enumerate((3, 200, 64)):
        for t in range(l):
            used[int(c.page_table[b, t // 16]), t % 16] = True
    c.k.masked_fill_(~used[:, None, :, None], math.nan)
    q[5:9] = math.nan
    out = torch.zeros_like(zero)
    kvd.paged_mass(c, q, lse, _starts(new), 8, 0.1, zero, out=out)
    assert torch.equal(out[0], want[0]) and torch.equal(out[2], want[2]) and out[1, 0, :200].isnan().all()
    c.page_table[2, 1] = -5
    c.t["status"].zero_()
    out = torch.zeros_like(zero)
    kvd.paged_mass(c, q, lse, _starts(new), 8, 0.1, zero, out=out)
    assert c.device_status() == 1
    assert torch.all(out[2, 0, 16:32] == 0) and torch.equal(out[2, 0, :16], want[2, 0, :16])
    assert torch.equal(out[2, 0, 32:], want[2, 0, 32:])


def test_mass_many_sequences():
    B = 300
    lens = [1 + (b * 37) % 300 for b in range(B)]
    new = [min(b % 4, lens[b]) for b in range(B)]
    c = _paged(kvd.F16, lens, 2, 64, 16, 8)
    _check(c, _q(sum(new), 4, 64, torch.float16, 9), new)


# --------------------------------------------------------------- eviction ---

def _evict(c, mass, keep, sink=0, recent=0, with_mass=True, spare=1):
    """Runs the call into fresh pages of the same pool (the last ones) and checks it."""
    B, heads, page = c.batch, LR.heads_of(c), c.page_size
    cols = (keep + page - 1) // page + spare
    to = (torch.arange(B * cols, device=DEV, dtype=torch.int32) + c.n_pages - B * cols).flip(0).view(B, cols)
    kept = torch.full((B, heads, keep), -9, dtype=torch.int32, device=DEV)
    lens = torch.full((B,), -9, dtype=torch.int32, device=DEV)
    mass_out = torch.full((B, heads, keep + 3), 7.0, device=DEV) if with_mass else None
    names = [n for n in ("rows", "k", "v", "k_scale", "v_scale") if n in c.t]
    before = {n: c.t[n].clone() for n in names}
    old = c.page_table.clone()
    kvd.paged_evict(c, mass, keep, to, kept, lens, mass_out=mass_out, sink=sink, recent=recent)
    assert c.device_status() == 0
    want = {n: before[n].clone() for n in names}
    for b in range(B):
        L = int(c.seq_lens[b])
        n = min(L, keep)
        assert int(lens[b]) == n
        r = torch.arange(n, device=DEV)
        for g in range(heads):
            ids = torch.tensor(LR.kept_of(mass[b, g], L, keep, sink, recent), dtype=torch.int64, device=DEV)
            assert torch.equal(kept[b, g, :n].long(), ids), (b, g)
            assert torch.all(kept[b, g, n:] == -9)
            if with_mass:
                assert torch.equal(mass_out[b, g, :n].nan_to_num(5.0), mass[b, g][ids].nan_to_num(5.0))
                assert torch.all(mass_out[b, g, n:] == 7.0)
            src, dst = old[b].long()[ids // page], to[b].long()[r // page]
            for name in names:
                x, y = before[name], want[name]
                if name == "rows":
                    y[dst, r % page] = x[src, ids % page]
                else:
                    y[dst, g, r % page] = x[src, g, ids % page]
    for name in names:
        assert torch.equal(want[name], c.t[name]), name
    return to, kept, lens, mass_out


def _room(make, lens, keep, page, *args, **kw):
    """A cache with spare pages at the pool's end for the rows that stay."""
    need = len(lens) * ((keep + page - 1) // page + 1)
    c = make(*args, **kw)
    t = dict(c.t)
    for n in ("rows", "k", "v", "k_scale", "v_scale"):
        if n in t:
            x = t[n]
            t[n] = torch.cat([x, x[:1].expand(need, *x.shape[1:]).clone()])
    if isinstance(c, kvd.LatentCache):
        new = kvd.LatentCache(c.dtype, c.batch, c.n_pages + need, page, c.max_pages, rank=c.rank,
                              rope_dim=c.rope_dim, tensors=t)
    else:
        new = kvd.PagedKVCache(c.dtype, c.batch, c.n_pages + need, c.n_kv_heads, page, c.max_pages,
                               head_dim=c.head_dim, tensors=t)
    new.len = c.len
    return new


def _masses(B, heads, n, seed):
    m = torch.randn(B, heads, n, generator=_gen(seed), device=DEV).mul_(2).exp_()
    return m.masked_fill_(torch.rand(m.shape, generator=_gen(seed + 1), device=DEV) < 0.2, 0.0)


@pytest.mark.parametrize("kind", [kvd.F16, kvd.BF16, kvd.INT8, "latent"])
@pytest.mark.parametrize("page,keep,sink,recent", [
    (16, 1, 0, 0), (16, 33, 4, 8), (48, 100, 0, 50), (64, 100, 100, 0), (64, 128, 28, 100), (128, 700, 4, 16)])
def test_evict(kind, page, keep, sink, recent):
    lens = [0, 1, keep, keep + 1, 3 * keep + 17, 650]
    lens[0] = 0
    if kind == "latent":
        c = _room(_latent, lens, keep, page, kvd.BF16, lens, page, keep, 128, 48)
    else:
        c = _room(_paged, lens, keep, page, kind, lens, 3, 64 if page == 16 else 128, page, keep)
    _evict(c, _masses(len(lens), LR.heads_of(c), c.len + 7, 3), keep, sink, recent)


@pytest.mark.parametrize("n,keep", [(5000, 1200), (17000, 16000), (140000, 3000), (200000, 150000)])
def test_evict_long(n, keep):
    """One block, several, and slices that no longer fit shared memory."""
    lens = [n, n // 3]
    c = _room(_paged, lens, keep, 64, kvd.INT8, lens, 1, 64, 64, 2)
    _evict(c, _masses(2, 1, c.len, 3), keep, 4, min(keep // 4, 1000))


def test_evict_ties_go_to_the_lower_index():
    lens = [9000, 9000, 300]
    c = _room(_paged, lens, 1000, 16, kvd.F16, lens, 2, 64, 16, 2)
    m = torch.zeros(3, 2, 9000, device=DEV)
    m[0, 1] = (torch.arange(9000, device=DEV) % 3).float()
    m[1, 0, 5000:] = -0.0
    m[1, 1, ::7] = 1e-42
    _evict(c, m, 1000, 3, 5)


def test_evict_unusual_weights():
    """Infinities, negative ones, NaN below all."""
    lens = [3000, 500]
    c = _room(_paged, lens, 400, 16, kvd.F16, lens, 2, 64, 16, 2)
    m = torch.randn(2, 2, 3000, generator=_gen(4), device=DEV)
    m[0, 0, ::5] = math.nan
    m[0, 1, 1::3] = math.inf
    m[1, 0, ::2] = -math.inf
    m[1, 1] = math.nan
    _evict(c, m, 400, 1, 1, with_mass=True)
    _evict(c, m, 400, 1, 1, with_mass=False)


def test_evict_strided_masses():
    lens = [700, 500]
    c = _room(_paged, lens, 64, 16, kvd.F16, lens, 2, 64, 16, 2)
    wide = _masses(2, 2, 1000, 5)
    _evict(c, wide[:, :, 100:900], 64)


def test_evict_reports_bad_pages_and_lengths():
    lens = [200, 200]
    c = _room(_paged, lens, 64, 16, kvd.F16, lens, 1, 64, 16, 2)
    m = _masses(2, 1, 200, 5)
    to, kept, _, _ = _evict(c, m, 64)
    for where in ("from", "to", "length"):
        c.t["status"].zero_()
        before = c.k.clone()
        table, dst = c.page_table.clone(), to.clone()
        j = int(kept[0, 0, 20]) // 16
        if where == "from":
            c.page_table[0, j] = c.n_pages
        elif where == "to":
            dst[0, 1] = -1
        else:
            c.seq_lens[1] = 10 ** 6
        k2, l2 = torch.zeros_like(kept), torch.zeros(2, dtype=torch.int32, device=DEV)
        kvd.paged_evict(c, m, 64, dst, k2, l2)
        assert c.device_status() == 1
        assert torch.equal(c.k, before)                # the same rows once more, or not at all
        assert torch.equal(k2, kept) and l2.tolist() == [64, 64]
        c.page_table.copy_(table)
        c.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))


@pytest.mark.parametrize("latent", [False, True])
def test_attend_accumulate_evict_and_go_on(latent):
    """As a server runs them: steps that count weights, an eviction, steps over what stays."""
    lens, keep, page, H = [300, 120], 96, 16, 8
    if latent:
        c = _room(_latent, lens, keep + 16, page, kvd.BF16, lens, page, 2, 128, 32, spare=2)
        D = 160
    else:
        c = _room(_paged, lens, keep + 16, page, kvd.BF16, lens, 2, 64, page, 2, spare=2)
        D = 64
    heads = LR.heads_of(c)
    mass = torch.zeros(2, heads, 400, device=DEV)
    want = torch.zeros(2, heads, 400, dtype=torch.float64, device=DEV)
    g = _gen(8)

    def step(c, mass):
        c.seq_lens += 1
        c.len = c.len + 1
        q = torch.randn(2, H, D, generator=g, device=DEV).bfloat16()
        row = torch.randn(2, 2 * D, generator=g, device=DEV).bfloat16()
        if latent:
            kvd.latent_append(c, row[:, :128], row[:, 128:160], _starts([1, 1]))
        else:
            kv = row.view(2, 2, D)
            kvd.paged_append(c, kv, kv, _starts([1, 1]))
        out, lse = _attend(c, q, [1, 1])
        ref = LR.attn(c, q, [0, 1, 2], c.seq_lens.tolist(), 0.1, 0, 0.95, mass.clone())
        LR.assert_close(out, ref["out"])
        kvd.paged_mass(c, q, lse, _starts([1, 1]), 1, 0.1, mass, decay=0.95)
        LR.assert_close(mass, ref["mass"])

    for _ in range(6):
        step(c, mass)
    to, kept, new_lens, new_mass = _evict(c, mass, keep, 4, 16)
    t = dict(c.t)
    t["page_table"], t["seq_lens"] = to, new_lens
    if latent:
        d = kvd.LatentCache(c.dtype, 2, c.n_pages, page, to.shape[1], rank=128, rope_dim=32, tensors=t)
    else:
        d = kvd.PagedKVCache(c.dtype, 2, c.n_pages, 2, page, to.shape[1], head_dim=64, tensors=t)
    d.len = keep
    grown = torch.zeros(2, heads, keep + 16, device=DEV)
    grown[:, :, :keep + 3] = new_mass
    for _ in range(6):
        step(d, grown)
    assert d.device_status() == 0


def test_mass_and_evict_in_a_graph_and_on_another_stream():
    lens = [900, 400]
    c = _room(_paged, lens, 128, 16, kvd.F16, lens, 2, 64, 16, 2)
    q = _q(2, 8, 64, torch.float16, 3)
    starts = _starts([1, 1])
    _, lse = _attend(c, q, [1, 1])
    mass = torch.zeros(2, 2, 900, device=DEV)
    kvd.paged_mass(c, q, lse, starts, 1, 0.1, mass)
    to, kept, new_lens, mass_out = _evict(c, mass, 128, 4, 8)
    m2, k2, l2, o2 = torch.zeros_like(mass), torch.zeros_like(kept), torch.zeros_like(new_lens), \
        torch.zeros_like(mass_out)
    zero = torch.zeros_like(mass)

    def both(stream=None):
        kvd.paged_mass(c, q, lse, starts, 1, 0.1, zero, out=m2, stream=stream)
        kvd.paged_evict(c, m2, 128, to, k2, l2, mass_out=o2, sink=4, recent=8, stream=stream)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    both(side)
    side.synchronize()
    assert torch.equal(k2, kept) and torch.equal(o2[:, :, :128], mass_out[:, :, :128])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    k2.zero_()
    m2.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(k2, kept) and torch.equal(m2[:, :, :400], mass[:, :, :400])


@pytest.mark.parametrize("dtype", [kvd.F16, kvd.BF16, kvd.INT8])
@pytest.mark.parametrize("H,Hkv,D,page,window", [(8, 2, 128, 16, 0), (14, 2, 64, 64, 200), (16, 1, 128, 128, 0),
                                                 (3, 3, 64, 32, 0), (32, 2, 128, 64, 129)])
def test_mass_of_many_rows(dtype, H, Hkv, D, page, window):
    """More rows than stay in shared memory: chunks of key tiles, rows that see some of them."""
    new, lens = [700, 1, 0, 400, 90], [2100, 900, 300, 400, 1500]
    c = _paged(dtype, lens, Hkv, D, page, 4)
    _check(c, _q(sum(new) + 2, H, D, X[dtype], 5), new, window=window)


def test_pools_above_32_bits():
    """Key-value pages at the end of a pool of more than 2^32 bytes a side."""
    page, D = 256, 128
    n_pages = (1 << 32) // (page * 2 * D * 2) + 20
    shape = (n_pages, 2, page, D)
    k, v = (torch.empty(shape, dtype=torch.float16, device=DEV) for _ in range(2))
    for i, x in enumerate((k, v)):
        x[-16:].copy_(torch.randn(16, 2, page, D, generator=_gen(i), device=DEV))
    table = (n_pages - 1 - torch.arange(12, device=DEV, dtype=torch.int32)).view(2, 6)
    lens = [1500, 300]
    c = kvd.PagedKVCache(kvd.F16, 2, n_pages, 2, page, 6, tensors={
        "k": k, "v": v, "page_table": table, "seq_lens": torch.tensor(lens, dtype=torch.int32, device=DEV)})
    c.len = 1500
    _check(c, _q(2, 8, D, torch.float16, 4), [1, 1])
    _check(c, _q(400, 8, D, torch.float16, 5), [300, 100])
    mass = _masses(2, 2, 1500, 3)
    to = (torch.arange(4, device=DEV, dtype=torch.int32) + n_pages - 16).view(2, 2)
    kept = torch.empty(2, 2, 300, dtype=torch.int32, device=DEV)
    new = torch.empty(2, dtype=torch.int32, device=DEV)
    kvd.paged_evict(c, mass, 300, to, kept, new, sink=2, recent=8)
    assert c.device_status() == 0
    for x in (k, v):
        for g in range(2):
            rows = x[table[0].long(), g].flatten(0, 1)
            assert torch.equal(x[to[0].long(), g].flatten(0, 1)[:300], rows[kept[0, g].long()])


def test_evict_of_sequences_that_share_pages():
    """Two sequences over the same first pages, and one table read twice by its heads: they keep what
    their own weights say, and the shared pages stay as they were."""
    lens = [200, 180]
    c = _room(_paged, lens, 64, 16, kvd.BF16, lens, 2, 64, 16, 2)
    c.page_table[1, :8] = c.page_table[0, :8]
    _evict(c, _masses(2, 2, 200, 5), 64, 4, 16)


def test_mass_of_a_nan_statistic_spoils_its_own_head_only():
    c = _paged(kvd.F16, [300, 300], 2, 64, 16, 2)
    q = _q(2, 8, 64, torch.float16, 3)
    _, lse = _attend(c, q, [1, 1])
    zero = torch.zeros(2, 2, 300, device=DEV)
    want, out = zero.clone(), zero.clone()
    kvd.paged_mass(c, q, lse, _starts([1, 1]), 1, 0.1, zero, out=want)
    lse[1, 5] = math.nan
    kvd.paged_mass(c, q, lse, _starts([1, 1]), 1, 0.1, zero, out=out)
    assert out[1, 1].isnan().all()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1, 0], want[1, 0])


def test_mass_of_an_empty_cache_and_of_lengths_out_of_range():
    c = _paged(kvd.F16, [40, 50], 2, 64, 16, 2)
    q = _q(2, 8, 64, torch.float16, 3)
    _, lse = _attend(c, q, [1, 1])
    mass = torch.ones(2, 2, 64, device=DEV)
    c.seq_lens.zero_()
    c.len = 0
    kvd.paged_mass(c, q, lse, _starts([1, 1]), 1, 0.1, mass, decay=0.5)
    assert torch.all(mass == 1.0)
    c.t["status"].zero_()
    c.seq_lens.copy_(torch.tensor([10 ** 6, -4]))
    c.len = 50
    kvd.paged_mass(c, q, lse, _starts([1, 1]), 1, 0.1, mass, decay=0.5)
    assert c.device_status() == 1
    assert torch.all(mass[1] == 1.0) and torch.all(mass[0, :, 50:] == 1.0) and torch.all(mass[0, :, :49] >= 0.5)
    kept = torch.full((2, 2, 5), -9, dtype=torch.int32, device=DEV)
    new = torch.full((2,), -9, dtype=torch.int32, device=DEV)
    c.seq_lens.zero_()
    c.len = 0
    kvd.paged_evict(c, mass, 5, torch.zeros(2, 1, dtype=torch.int32, device=DEV), kept, new)
    assert new.tolist() == [0, 0] and torch.all(kept == -9)


@pytest.mark.parametrize("latent", [False, True])
def test_runs_longer_than_told(latent):
    """More new tokens in a sequence than max_new: reported, and the first max_new are counted."""
    if latent:
        c, D, scale = _latent(kvd.BF16, [100, 400], 16, 2, 128, 32), 160, 0.1
    else:
        c, D, scale = _paged(kvd.BF16, [100, 400], 1, 64, 16, 2), 64, 0.1
    q = _q(30, 4, D, torch.bfloat16, 3)
    _, lse = _attend(c, q, [10, 20], 0, scale)
    mass = torch.zeros(2, 1, 400, device=DEV)
    kvd.paged_mass(c, q, lse, _starts([10, 20]), 12, scale, mass)
    assert c.device_status() == 1
    full = LR.attn(c, q, [0, 10, 30], [100, 400], scale, 0, 1.0, torch.zeros_like(mass))["mass"]
    LR.assert_close(mass[0], (full[0][0], full[1][0]))
    assert abs(float(mass[1].double().sum()) - 12 * 4) < 12 * 4 * 2 * D * 2.0 ** -23 * 64


@pytest.mark.parametrize("latent", [False, True])
def test_a_batch_without_new_tokens(latent):
    """Steps whose batch is empty: attention with statistics is a no-op, the weights only decay."""
    c, D = (_latent(kvd.BF16, [100, 40], 16, 2, 128, 32), 160) if latent else \
        (_paged(kvd.BF16, [100, 40], 2, 64, 16, 2), 64)
    heads, V = LR.heads_of(c), 128 if latent else 64
    q = torch.empty(0, 8, D, dtype=torch.bfloat16, device=DEV)
    out, lse = torch.empty(0, 8, V, dtype=torch.bfloat16, device=DEV), torch.empty(0, 8, device=DEV)
    make, attend = (kvd.make_latent_workspace, kvd.latent_attn) if latent else (kvd.make_paged_workspace, kvd.paged_attn)
    ws = make(c, 8, 1, 1)
    for max_new in (0, 1):
        attend(c, q, _starts([0, 0]), max_new, 0.1, out, ws, lse=lse)
        mass = torch.ones(2, heads, 100, device=DEV)
        kvd.paged_mass(c, q, lse, _starts([0, 0]), max_new, 0.1, mass, decay=0.5)
        assert torch.all(mass[0] == 0.5) and torch.all(mass[1, :, :40] == 0.5) and torch.all(mass[1, :, 40:] == 1.0)
    assert c.device_status() == 0


@pytest.mark.parametrize("kind", ["paged", "latent", "latent, dense queries"])
def test_rotated_tokens_behind_an_eviction(kind):
    """After an eviction a token's position is not its place: qk_norm_rope rotates by the position and the
    append takes rows as they are.  The latent cache's parts of heads go through it as rows of one head."""
    lens, keep, page, H, T, P = [300, 120], 96, 16, 6, 2, 32
    latent = kind != "paged"
    if latent:
        c = _room(_latent, lens, keep + 16, page, kvd.BF16, lens, page, 2, 128, P)
    else:
        c = _room(_paged, lens, keep + 16, page, kvd.BF16, lens, 2, 64, page, 2)
    heads = LR.heads_of(c)
    to, _, new_lens, _ = _evict(c, _masses(2, heads, 300, 3), keep, 4, 16)
    t = dict(c.t, page_table=to, seq_lens=new_lens)
    if latent:
        d = kvd.LatentCache(c.dtype, 2, c.n_pages, page, to.shape[1], rank=128, rope_dim=P, tensors=t)
    else:
        d = kvd.PagedKVCache(c.dtype, 2, c.n_pages, 2, page, to.shape[1], head_dim=64, tensors=t)
    d.len = keep
    f, m = R.freqs(P, 10000.0)
    rope = kvd.rope_table(P)
    g = _gen(9)
    positions = torch.tensor(lens, dtype=torch.int32, device=DEV)       # of the next tokens, not their places
    place = torch.arange(2, device=DEV)
    for _ in range(3):
        d.seq_lens += 1
        d.len = d.len + 1
        at = (d.seq_lens - 1).long()
        ids, in_page = to[place, at // page].long(), at % page
        w = torch.rand(128 if latent else 64, generator=g, device=DEV) + 0.5
        if latent:
            down = torch.randn(T, 128 + P, generator=g, device=DEV).bfloat16()
            wide = torch.randn(T, H, 64 + P, generator=g, device=DEV).bfloat16()
            q_pe = wide[:, :, 64:].contiguous() if kind != "latent" else wide[:, :, 64:]
            q = torch.randn(T, H, 128 + P, generator=g, device=DEV).bfloat16()
            absorbed = q[:, :, :128].clone()
            k_rot = torch.empty(T, 1, P, device=DEV, dtype=torch.bfloat16)
            kvd.qk_norm_rope(down[:, 128:][:, None], None, positions, rope, k_rot, None)
            kvd.qk_norm_rope(q_pe.flatten(0, 1)[:, None], None, positions.repeat_interleave(H), rope,
                             q.view(-1, 1, 128 + P)[..., 128:], None)
            assert torch.equal(q[:, :, :128], absorbed)
            kvd.latent_append(d, down[:, :128], k_rot[:, 0], _starts([1, 1]), c_weight=w)
            y, err = R.turned(q_pe, positions, f, m, False)
            R.assert_within(q[:, :, 128:], y, R.rounding(y, err, q.dtype), "q")
            y, err = R.turned(down[:, None, :128], positions, None, 1.0, False, w)
            got = d.rows[ids, in_page]
            R.assert_within(got[:, :128], y[:, 0], R.rounding(y, err, q.dtype)[:, 0], "latent")
            y, err = R.turned(down[:, None, 128:], positions, f, m, False)
            R.assert_within(got[:, 128:], y[:, 0], R.rounding(y, err, q.dtype)[:, 0], "key part")
        else:
            qkv = torch.randn(T, H + 4, 64, generator=g, device=DEV).bfloat16()
            q, k, v = torch.empty_like(qkv[:, :H]), torch.empty_like(qkv[:, :2]), qkv[:, H + 2:]
            kvd.qk_norm_rope(qkv[:, :H], qkv[:, H:H + 2], positions, rope, q, k, w, w)
            kvd.paged_append(d, k, v, _starts([1, 1]))
            y, err = R.turned(qkv[:, H:H + 2], positions, f, m, False, w)
            R.assert_within(d.k[ids, :, in_page], y, R.rounding(y, err, q.dtype), "key")
            assert torch.equal(d.v[ids, :, in_page], v)
        out, lse = _attend(d, q, [1, 1], window=40)                      # the last 40 that stayed
        want = LR.attn(d, q, [0, 1, 2], d.seq_lens.tolist(), 0.1, 40)
        LR.assert_close(out, want["out"])
        LR.assert_close(lse, want["lse"])
        positions += 1
    assert d.device_status() == 0
