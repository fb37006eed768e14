"""kvd_paged_attn where values are not tame: NaN and infinite queries, one key with nearly all the
weight, value scales of very different size, and neighbours whose rows share a tile."""
import math

import pytest
import torch

import long_context_decode_kv_gb300 as kvd
import paged_ref as R
from test_gpu_paged import DEV, X, _attend, _cache, _q, _starts

pytestmark = pytest.mark.gpu
# new tokens and length of one sequence of 4 heads a KV head: the kernel for few rows, 128 rows and
# row tiles in pairs, each with its item whole and cut between CTAs
SHAPES = [(1, 60), (1, 30000), (8, 300), (8, 20000), (20, 100), (20, 9000), (300, 400), (300, 9000)]


def _x(dtype):
    return X.get(dtype, torch.bfloat16)


# ------------------------------------------------------- NaN and infinities ---

@pytest.mark.parametrize("dtype", [kvd.F16, kvd.BF16, kvd.INT8])
@pytest.mark.parametrize("new,L", SHAPES)
def test_a_query_that_is_not_finite_gives_a_nan_row(dtype, new, L):
    """And leaves the others as they are, wherever the item is cut."""
    c = _cache(dtype, [L], 2, 128, 64, L)
    q = _q(new, 8, 128, _x(dtype), new)
    q[0, 1, 5] = math.nan
    q[new // 2, 6, 127] = math.inf
    q[new - 1, 3] = math.nan
    out = _attend(c, q, [new])
    want, tol = R.attn_ref(c, q, [0, new], [L], 128 ** -0.5)
    bad = ~torch.isfinite(q).all(-1)
    assert bool(torch.isnan(out[bad]).all())
    R.assert_within(out[~bad], want[~bad], tol[~bad])
    assert c.device_status() == 0


# --------------------------------------------------------------- neighbours ---

@pytest.mark.parametrize("dtype", [kvd.F16, kvd.BF16, kvd.INT8])
@pytest.mark.parametrize("G,new", [(4, [1, 8]), (7, [2, 4]), (4, [9, 30]), (7, [5, 18]), (4, [20, 200]),
                                   (3, [50, 300]), (7, [25, 90])])
def test_a_sequence_does_not_depend_on_its_neighbour(dtype, G, new):
    """The tile's rows behind a sequence's last are the next one's queries, or none's."""
    c = _cache(dtype, [2000, 2300], 2, 128, 64, G)
    q = _q(sum(new), 2 * G, 128, _x(dtype), G)
    n = new[0]
    first = _attend(c, q, new)[:n]
    for other in (300.0, 0.0, math.nan):
        p = q.clone()
        p[n:] *= other
        assert torch.equal(_attend(c, p, new)[:n], first)


@pytest.mark.parametrize("dtype", [kvd.F16, kvd.BF16, kvd.INT8])
@pytest.mark.parametrize("G,new", [(7, 4), (4, 20), (3, 11), (7, 200), (6, 300)])
def test_a_call_does_not_depend_on_the_one_before(dtype, G, new):
    """Rows of a tile that hold no query, after calls whose queries filled them with large values."""
    c = _cache(dtype, [3000], 2, 128, 64, G + new)
    q = _q(new, 2 * G, 128, _x(dtype), new)
    first = _attend(c, q, [new])
    for scale in (1e3, math.nan):
        for g, n in ((G, new), (8, 16), (8, 200), (16, 2)):
            _attend(c, torch.full((n, 2 * g, 128), scale, dtype=q.dtype, device=DEV), [n])
        assert torch.equal(_attend(c, q, [new]), first)


# ------------------------------------------------ weights of very different size ---

U16 = 2.0 ** -11            # f16: half a step of a weight, relative; 2^-25 below 2^-14
# Binary places above 1 that a row's largest weight takes, so that small ones keep as many more
# (int8: of the product with the value's scale, which may be half of the unit it is counted in).
REACH = {kvd.F16: 6, kvd.INT8: 4}


def _set_rows(c, b, name, values, scale=None):
    """Tokens [0, n) of sequence b, every KV head: values [n, D] (int8: codes, with scales [n])."""
    n = values.shape[0]
    p = torch.arange(n, device=DEV)
    page, off = c.page_table[b, p // c.page_size].long(), p % c.page_size
    c.t[name][page, :, off] = values[:, None].to(c.t[name].dtype)
    if scale is not None:
        c.t[name + "_scale"][page, :, off] = scale[:, None].float()


def _few_channels(c, b, L, z, v, v_scale):
    """A cache whose logits are z[t] (through channel 0 of a query of ones) and whose values are v[t]."""
    k = torch.zeros(L, c.head_dim, device=DEV)
    if c.dtype == kvd.INT8:
        k[:, 0] = torch.where(z == 0, 0.0, 127.0 * z.sign())
        _set_rows(c, b, "k", k, torch.where(z == 0, 1.0, z.abs() / 127).float())
        _set_rows(c, b, "v", v, v_scale)
    else:
        k[:, 0] = z
        _set_rows(c, b, "k", k)
        _set_rows(c, b, "v", v * v_scale[:, None])


@pytest.mark.parametrize("dtype,x", [(kvd.F16, torch.float16), (kvd.INT8, torch.float16),
                                     (kvd.INT8, torch.bfloat16)])
@pytest.mark.parametrize("new,L", SHAPES)
@pytest.mark.parametrize("at", [0, 40, 390])
@pytest.mark.parametrize("below", [22.4, 25.6])
def test_one_key_holds_nearly_all_the_weight(dtype, x, new, L, at, below):
    """The others are 2^-below of it each.  Its value is zero, so that theirs is what comes out.

    A weight is off by half a step (2^-11 of it), or below f16's normal numbers by 2^-25 of
    their reference, which lies REACH places below the row's largest weight; by its logit (2^-22
    of it, and the exponential's 2^-22); the sums and the output add their own."""
    if L <= at:
        pytest.skip("the key lies behind the sequence")
    D = 128
    c = _cache(dtype, [L], 2, D, 64, L)
    z = torch.zeros(L, device=DEV)
    z[at] = 16.0
    v = torch.full((L, D), 127.0, device=DEV)
    v[at] = 0.0
    _few_channels(c, 0, L, z, v, torch.full((L,), 8.0, device=DEV))
    q = torch.zeros(new, 8, D, dtype=x, device=DEV)
    q[..., 0] = 1.0
    scale = below * math.log(2) / 16
    out = _attend(c, q, [new], scale=scale).double()
    p = torch.arange(L - new, L, device=DEV).double()
    rest = torch.where(p >= at, p, p + 1)                  # keys beside it that a token sees
    w = torch.where(p >= at, 2.0 ** -below, 1.0)
    want = 1016 * rest * w / (rest * w + (p >= at))
    off = torch.where(p >= at, 2.0 ** (-25 - REACH[dtype]) / w, 0.0)
    err = want * (off.clamp_min(U16) + below * 2.0 ** -22 + (rest / 8 + 64) * 2.0 ** -23) * 1.01
    tol = R.rounding(want, err, x)
    R.assert_within(out, want[:, None, None].expand_as(out), tol[:, None, None].expand_as(out))
    assert c.device_status() == 0


def test_an_attention_sink_over_a_long_cache():
    """131,072 keys, the first with 0.9 or 0.99 of the weight: what is left of the others' weights."""
    D, L = 128, 131072
    c = _cache(kvd.F16, [L], 1, D, 64, 9)
    q = torch.zeros(1, 4, D, dtype=torch.float16, device=DEV)
    q[..., 0] = 1.0
    g = torch.Generator(device=DEV).manual_seed(10)
    for share in (0.9, 0.99):
        z = torch.randn(L, generator=g, device=DEV).half().float()
        z[0] = 0.0
        z[0] = float((z[1:].double().exp().sum() * share / (1 - share)).log())
        z = z.half().float()
        v = (torch.randn(L, D, generator=g, device=DEV) + 0.3).half().float()
        _few_channels(c, 0, L, z, v, torch.ones(L, device=DEV))
        out = _attend(c, q, [1], scale=1.0)[0].double()
        w = torch.softmax(z.double(), 0)
        want = w @ v.double()
        # each weight's rounding taken as independent of the others': six deviations of their sum
        step = torch.maximum(w * U16, 2.0 ** -25 / 2 ** REACH[kvd.F16] * w.max())
        err = 6 * (step.square() @ v.double().square()).sqrt() / 3 ** 0.5
        # logits, exponentials, and the running sums of 16 keys a step in the longest piece
        err = err + (w @ v.double().abs()) * (32 * 2.0 ** -22 + (L / 152 / 8 + 512) * 2.0 ** -23)
        R.assert_within(out, want.expand(4, D), R.rounding(want, err, torch.float16).expand(4, D))


@pytest.mark.parametrize("x", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("new,L", [s for s in SHAPES if s[1] >= 300])
@pytest.mark.parametrize("at", [0, 200])
@pytest.mark.parametrize("places", [12, 24])
def test_one_large_value_scale_on_a_key_without_weight(x, new, L, at, places):
    """Its scale is 2^places of the others', and its weight 2^-100: only the keys of its own tile
    may lose what f16 cannot hold beside it.

    A product of weight and scale is off by half a step, or by 2^-25 in units of at most 64 times
    the tile's largest scale (the unit is the power of two above that, or up to 2^5 of it before
    it falls)."""
    D = 128
    c = _cache(kvd.INT8, [L], 2, D, 64, L)
    g = torch.Generator(device=DEV).manual_seed(L + at)
    z = torch.zeros(L, device=DEV)
    z[at] = -100.0
    v = torch.randint(64, 128, (L, D), generator=g, device=DEV).float()
    vs = torch.rand(L, generator=g, device=DEV) * 0.5 + 0.5
    vs[at] *= 2.0 ** places
    _few_channels(c, 0, L, z, v, vs)
    q = torch.zeros(new, 8, D, dtype=x, device=DEV)
    q[..., 0] = 1.0
    out = _attend(c, q, [new], scale=math.log(2)).double()
    p = torch.arange(L - new, L, device=DEV)
    t = torch.arange(L, device=DEV)
    w = ((t <= p[:, None]) & (t != at)).double()
    l = w.sum(-1, keepdim=True)
    top = torch.stack([s.max() for s in vs.split(128)]).repeat_interleave(128)[:L].double()
    val = v.double() * vs.double()[:, None]
    want = w @ val / l
    step = torch.maximum(U16 * vs.double(), 2.0 ** (-25 - REACH[kvd.INT8]) * 64 * top)
    err = w @ (v.double() * step[:, None]) / l
    err = err + want * ((l / 8 + 64) * 2.0 ** -23) * 1.01
    want, tol = (a[:, None].expand_as(out) for a in (want, R.rounding(want, err, x)))
    R.assert_within(out, want, tol)
    assert c.device_status() == 0


# ------------------------------------------------------------- rows of no sequence ---

@pytest.mark.parametrize("dtype", [kvd.F16, kvd.INT8])
@pytest.mark.parametrize("first,new", [(3, [2, 4]), (1, [1, 1, 1]), (70, [90, 0, 5]), (200, [1])])
def test_rows_before_the_first_sequence_count_for_nothing(dtype, first, new):
    """starts[0] above 0: a part of a larger batch's rows, and nothing to report."""
    H, Hkv, D, T = 8, 2, 64, first + sum(new) + 2
    lens = [n + 30 * b for b, n in enumerate(new)]
    c = _cache(dtype, lens, Hkv, D, 16, first)
    before = {n: c.t[n].clone() for n in ("k", "v")}
    starts = _starts(new) + first
    x = _q(T, H + 2 * Hkv, D, torch.float16, first)
    q_out, out = (torch.full((T, H, D), 7.0, dtype=x.dtype, device=DEV) for _ in range(2))
    kvd.paged_append(c, x[:, H:H + Hkv], x[:, H + Hkv:], starts, q=x[:, :H], q_out=q_out)
    kvd.paged_attn(c, q_out, starts, max(new), 0.125, out, kvd.make_paged_workspace(c, H, T, max(new)))
    assert c.device_status() == 0
    rows = slice(first, first + sum(new))
    assert torch.equal(q_out[rows], x[rows, :H])
    want, tol = R.attn_ref(c, q_out, starts.tolist(), lens, 0.125)
    R.assert_within(out[rows], want[rows], tol[rows])
    for o in (q_out, out):
        assert torch.all(o[:first] == 7.0) and torch.all(o[first + sum(new):] == 7.0)
    assert int((c.k != before["k"]).any(-1).any(1).sum()) <= sum(new)


# --------------------------------------------------------------- long among many ---

@pytest.mark.parametrize("dtype", [kvd.F16, kvd.INT8])
@pytest.mark.parametrize("window", [0, 100])
@pytest.mark.parametrize("B,chunks", [(49, {0: 1100}), (50, {49: 1500, 20: 600}), (700, {3: 900, 31: 1025, 650: 1300})])
def test_long_chunks_among_many_sequences(dtype, window, B, chunks):
    """More sequences than are counted a warp each, some with more row tiles than a lane counts alone."""
    lens = [1 + b * 29 % 200 for b in range(B)]
    new = [b % 2 for b in range(B)]
    for b, n in chunks.items():
        lens[b], new[b] = n + 77, n
    c = _cache(dtype, lens, 1, 64, 32, B)
    q = _q(sum(new), 8, 64, torch.float16, B)
    out = _attend(c, q, new, window)
    want, tol = R.attn_ref(c, q, _starts(new).tolist(), lens, 0.125, window)
    R.assert_within(out, want, tol)
    assert c.device_status() == 0


# ----------------------------------------------------------- scales of all sizes ---

@pytest.mark.parametrize("x", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("new,L", SHAPES)
@pytest.mark.parametrize("places", [1, 3, 8])
@pytest.mark.parametrize("window", [0, 150])
def test_value_scales_of_all_sizes(x, new, L, places, window):
    """Scales spread over several times 2^places, a tenth of them zero, within the header's bound:
    weight times scale to 2^-11, and to 2^-24 of the row's largest weight times the largest scale
    of the 128 keys around; logits and sums as in attn_ref."""
    D, H, Hkv = 64, 8, 2
    c = _cache(kvd.INT8, [L], Hkv, D, 16, L + places)
    g = torch.Generator(device=DEV).manual_seed(L + places)
    e = (torch.randn(c.v_scale.shape, generator=g, device=DEV) * places).clamp(-30, 30)
    c.v_scale.copy_(torch.exp2(e - e.max() + 8))      # values stay in f16's range
    c.v_scale[torch.rand(e.shape, generator=g, device=DEV) < 0.1] = 0.0
    q = _q(new, H, D, x, new)
    out = _attend(c, q, [new], window).double()
    p = torch.arange(L - new, L, device=DEV)[:, None]
    t = torch.arange(L, device=DEV)
    seen = (t <= p) & ((t > p - window) | (window == 0))
    first = max(0, L - new - window + 1) if window else 0  # before it no row sees a key
    for h in range(H):
        k, v, ks, vs = (R.rows_of(c.t[n], c.page_table[0], L, h // (H // Hkv)).double()
                        for n in ("k", "v", "k_scale", "v_scale"))
        k = k * ks[:, None]
        qq = q[:, h].double() * D ** -0.5
        z = torch.where(seen, qq @ k.T, -math.inf)
        w = torch.softmax(z, -1)
        near = torch.where(t < first, 0.0, vs)
        near = torch.stack([s.max() for s in near.split(128)]).repeat_interleave(128)[:L]
        step = torch.maximum(U16 * w * vs, 2.0 ** -24 * seen * w.amax(-1, keepdim=True) * near)
        mag = torch.where(seen, qq.abs() @ k.abs().T, 0.0).amax(-1, keepdim=True)
        n = seen.sum(-1, keepdim=True).double()
        rest = 2 * D * 2.0 ** -23 * mag + (n / 8 + 64) * 2.0 ** -23
        want = w @ (v * vs[:, None])
        err = (step @ v.abs() + (w @ (v.abs() * vs[:, None])) * rest) * 1.01
        R.assert_within(out[:, h], want, R.rounding(want, err, x), f"head {h}")
    assert c.device_status() == 0
