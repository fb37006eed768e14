"""kvd_qk_norm_rope against the 64-bit definition (bounds in paged_ref.py)."""
import pytest
import torch

import long_context_decode_kv_gb300 as kvd
import paged_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _case(T, H, Hkv, D, x, seed, pad=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    qkv = (torch.randn(T, H + 2 * Hkv + pad, D, generator=g, device=DEV) * 2).to(x)
    w = [torch.rand(D, generator=g, device=DEV) + 0.5 for _ in range(2)]
    return qkv[:, :H], qkv[:, H:H + Hkv], w


def _check(q, k, pos, rope_args, q_out, k_out, w=(None, None), eps=1e-6, table=True):
    rot, inter, scaling, factor, orig = rope_args
    f, m = R.freqs(rot, 10000.0, scaling, factor, orig) if table else (None, 1.0)
    t = kvd.rope_table(rot, interleaved=inter, scaling=scaling, factor=factor, orig_len=orig) \
        if table else None
    want = [R.turned(a, pos, f, m, inter, ww, eps) if a is not None else None
            for a, ww in ((q, w[0]), (k, w[1]))]
    kvd.qk_norm_rope(q, k, pos if table else None, t, q_out, k_out, q_weight=w[0], k_weight=w[1], eps=eps)
    for got, ref, name in ((q_out, want[0], "q"), (k_out, want[1], "k")):
        if ref is not None:
            y, err = ref
            R.assert_within(got, y, R.rounding(y, err, got.dtype), name)


@pytest.mark.parametrize("x", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("D,rot", [(16, 16), (48, 32), (64, 64), (64, 16), (80, 48), (128, 128), (128, 32),
                                   (192, 64), (256, 256), (272, 272), (512, 128), (1024, 1024)])
def test_types_layouts_and_head_dims(x, inter, norm, D, rot):
    T, H, Hkv = 5, 6, 2
    q, k, w = _case(T, H, Hkv, D, x, D + rot)
    pos = torch.tensor([0, 1, 777, 131071, 1000003], dtype=torch.int32, device=DEV)
    _check(q, k, pos, (rot, inter, "none", 1, 0), torch.empty(T, H, D, dtype=x, device=DEV),
           torch.empty(T, Hkv, D, dtype=x, device=DEV), w if norm else (None, None))


@pytest.mark.parametrize("x", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("out", [torch.float16, torch.bfloat16, torch.float32])
def test_output_types(x, out):
    q, k, w = _case(3, 4, 4, 128, x, 5)
    pos = torch.arange(3, dtype=torch.int32, device=DEV) + 4000
    _check(q, k, pos, (128, False, "none", 1, 0), torch.empty(3, 4, 128, dtype=out, device=DEV),
           torch.empty(3, 4, 128, dtype=torch.float16, device=DEV), w)


@pytest.mark.parametrize("scaling,factor,orig", [("linear", 4, 0), ("ntk", 8, 0), ("yarn", 16, 8192),
                                                 ("bands", 8, 8192)])
@pytest.mark.parametrize("T,H,Hkv", [(1, 1, 1), (1, 32, 8), (7, 33, 3), (300, 5, 1), (1300, 16, 2)])
def test_scalings_and_sizes(scaling, factor, orig, T, H, Hkv):
    q, k, w = _case(T, H, Hkv, 64, torch.bfloat16, T + H)
    pos = (torch.arange(T, device=DEV) * 37 + 2 ** 31 - 1 - 37 * T).int()   # up to the last positions
    _check(q, k, pos, (64, T % 2 == 0, scaling, factor, orig),
           torch.empty(T, H, 64, dtype=torch.float32, device=DEV),
           torch.empty(T, Hkv, 64, dtype=torch.bfloat16, device=DEV), w)


def test_norm_alone_queries_alone_and_one_weight():
    q, k, w = _case(4, 3, 2, 128, torch.float16, 9)
    pos = torch.zeros(4, dtype=torch.int32, device=DEV)
    _check(q, k, pos, (128, False, "none", 1, 0), torch.empty_like(q), torch.empty_like(k), w, table=False)
    _check(q, None, pos + 9, (128, False, "none", 1, 0), torch.empty_like(q), None, (w[0], None))
    _check(q, k, pos + 9, (64, True, "none", 1, 0), torch.empty_like(q), torch.empty_like(k), (None, w[1]))


def test_zero_rows_and_tiny_values():
    q, k, w = _case(2, 2, 2, 128, torch.float32, 11)
    q, k = q * 0, k * 1e-12
    pos = torch.tensor([3, 4], dtype=torch.int32, device=DEV)
    _check(q, k, pos, (128, False, "none", 1, 0), torch.empty(2, 2, 128, device=DEV),
           torch.empty(2, 2, 128, device=DEV), w)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D", [64, 128, 512])
def test_in_place_in_a_fused_projection_and_nothing_else_written(inter, D):
    T, H, Hkv = 9, 5, 2
    x = torch.randn(T, H + 2 * Hkv + 1, D, device=DEV, dtype=torch.bfloat16)
    before = x.clone()
    q, k = x[:, :H], x[:, H:H + Hkv]
    pos = torch.arange(T, dtype=torch.int32, device=DEV) * 11
    f, m = R.freqs(D)
    want = [R.turned(a, pos, f, m, inter) for a in (before[:, :H], before[:, H:H + Hkv])]
    kvd.qk_norm_rope(q, k, pos, kvd.rope_table(D, interleaved=inter), q, k)
    for got, (y, err) in zip((q, k), want):
        R.assert_within(got, y, R.rounding(y, err, got.dtype))
    assert torch.equal(x[:, H + Hkv:], before[:, H + Hkv:])


def test_no_tokens_and_another_stream():
    t = kvd.rope_table(64)
    e = torch.empty(0, 4, 64, device=DEV)
    kvd.qk_norm_rope(e, None, torch.empty(0, dtype=torch.int32, device=DEV), t, e, None)
    q = torch.randn(3, 4, 64, device=DEV)
    out = torch.empty_like(q)
    pos = torch.arange(3, dtype=torch.int32, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    kvd.qk_norm_rope(q, None, pos, t, out, None, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    y, err = R.turned(q, pos, *R.freqs(64), False)
    R.assert_within(out, y, R.rounding(y, err, out.dtype))


def test_feeds_the_decode_step():
    """Normed, rotated tokens one after the other through decode_step, against attention in 64 bits."""
    H, Hkv, D, L = 8, 2, 128, 150
    q, k, w = _case(L, H, Hkv, D, torch.float16, 21)
    v = torch.randn(L, Hkv, D, device=DEV).half()
    pos = torch.arange(L, dtype=torch.int32, device=DEV)
    t = kvd.rope_table(128)
    qo = torch.empty(L, H, D, device=DEV)
    ko = torch.empty(L, Hkv, D, device=DEV, dtype=torch.float16)
    kvd.qk_norm_rope(q, k, pos, t, qo, ko, q_weight=w[0], k_weight=w[1])
    cache = kvd.KVCache(kvd.F16, 1, Hkv, 256)
    kvd.kv_append(cache, ko[None, :L - 1].contiguous(), v[None, :L - 1].contiguous())
    ws = kvd.make_workspace(cache, H)
    out = torch.empty(1, H, D, device=DEV)
    kvd.decode_step(cache, qo[L - 1:], ko[None, L - 1:], v[None, L - 1:], D ** -0.5, -1, 0, 0, out, ws)
    f, m = R.freqs(128)
    yq = R.turned(q[L - 1:], pos[L - 1:], f, m, False, w[0])[0]
    yk = ko.double()
    for h in range(H):
        p = torch.softmax(yk[:, h // 4] @ yq[0, h] * D ** -0.5, 0)
        ref = p @ v[:, h // 4].double()
        assert (out[0, h] - ref).norm() <= 1e-4 * ref.norm()
