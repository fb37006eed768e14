"""Host side of the norm/rotation and paged-cache calls: frequencies against their
definitions, refusals, and the binding's checks.  No GPU."""
import ctypes as C
import math
from fractions import Fraction

import pytest
import torch

import long_context_decode_kv_gb300 as kvd
import paged_ref as R

OK, INVALID, UNSUPPORTED, CAPACITY, CUDA, TIMEOUT, WORKSPACE = range(7)
FAKE = 0x7f0000000000  # aligned, never dereferenced on the host


@pytest.fixture(scope="module", autouse=True)
def _built():
    from long_context_decode_kv_gb300 import build
    build.build()


@pytest.mark.parametrize("rot", [16, 32, 48, 64, 128, 256])
@pytest.mark.parametrize("scaling,factor,orig,low,high", [
    ("none", 1, 0, 0, 0), ("linear", 4, 0, 0, 0), ("ntk", 8, 0, 0, 0), ("yarn", 8, 8192, 0, 0),
    ("yarn", 32, 32768, 2, 16), ("bands", 8, 8192, 0, 0), ("bands", 2.5, 4096, 0, 9), ("yarn", 1, 1, 0, 0)])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_freqs_match_their_definitions(rot, scaling, factor, orig, low, high, base):
    t = kvd.rope_table(rot, base, scaling=scaling, factor=factor, orig_len=orig, low=low, high=high,
                       device="cpu")
    f, m = R.freqs(rot, base, scaling, factor, orig, low, high)
    turns = t.freqs.double() * 2.0 ** -64
    # a few roundings of 2^-53 (power, product, quotient), and half a step of the word
    assert torch.all((turns * 2 * math.pi - f).abs() <= f * 2.0 ** -48 + 2.0 ** -61)
    assert abs(t.mscale - m) <= m * 2.0 ** -24
    assert t.freqs.numel() == rot // 2 and bool((t.freqs > 0).all())


def test_far_positions_keep_their_angle():
    t = kvd.rope_table(128, device="cpu")
    for i, word in enumerate(t.freqs.tolist()):
        f = Fraction(10000.0 ** (-2.0 * i / 128)) / Fraction(2 * math.pi)
        for p in (1, 8191, 1 << 20, (1 << 31) - 1):
            got = Fraction((p * word) % (1 << 64), 1 << 64)
            off = abs((got - p * f) - round(got - p * f))
            # the word is off by half a step and the 64-bit formula by 2^-50 of f
            assert off <= p * (Fraction(1, 1 << 64) + f * Fraction(1, 1 << 50))


def test_freqs_refusals():
    L = kvd.lib()
    buf, m = (C.c_uint64 * 512)(), C.c_float()

    def call(rot=64, base=1e4, scaling=0, factor=1.0, orig=4096.0, low=0.0, high=0.0, out=buf):
        return L.kvd_rope_freqs(rot, base, scaling, factor, orig, low, high, out, C.byref(m))

    assert call() == OK
    for rot in (0, -16, 8, 24, 1040):
        assert call(rot=rot) == INVALID
    for base in (1.0, 0.0, -5.0, math.nan, math.inf):
        assert call(base=base) == INVALID
    assert call(scaling=5) == INVALID and call(scaling=-1) == INVALID
    assert call(scaling=1, factor=0.5) == INVALID
    assert call(scaling=1, factor=math.nan) == INVALID
    assert call(scaling=0, factor=0.5) == OK        # ignored without a stretch
    assert call(scaling=3, orig=0.0) == INVALID
    assert call(scaling=4, low=4.0, high=1.0) == INVALID
    assert call(scaling=3, low=0.0, high=8.0) == INVALID
    assert call(scaling=4, low=0.0, high=8.0) == OK
    assert call(out=None) == INVALID
    with pytest.raises(ValueError):
        kvd.rope_table(64, scaling="cubic", device="cpu")
    with pytest.raises(kvd.KvdError):
        kvd.rope_table(20, device="cpu")


def _h(x=FAKE, n=8, D=128, dtype=0, stride=None):
    return kvd.HeadsStruct(x, n * D if stride is None else stride, dtype, n)


def _rope(freqs=FAKE, rot=64, inter=0, m=1.0, reserved=0):
    return kvd.RopeStruct(freqs, rot, inter, m, reserved)


def test_qk_norm_rope_refusals():
    f = kvd.lib().kvd_qk_norm_rope

    def call(q=None, qo=None, k=None, ko=None, n=4, D=128, pos=FAKE, rope=_rope(), qw=None, kw=None,
             eps=1e-6):
        return f(q or _h(n=32), qo or _h(FAKE + (1 << 30), n=32), k, ko, n, D, pos, rope, qw, kw, eps,
                 None)

    assert call(n=0) == OK
    assert call(n=-1) == INVALID
    assert call(D=72) == UNSUPPORTED and call(D=1040) == UNSUPPORTED and call(D=0) == UNSUPPORTED
    assert call(q=_h(FAKE + 2, 32)) == INVALID
    assert call(q=_h(None, 32)) == INVALID
    assert call(q=_h(n=32, dtype=3)) == INVALID
    assert call(q=_h(n=0)) == INVALID
    assert call(q=_h(n=32, stride=32 * 128 - 8)) == INVALID      # tokens overlap
    assert call(q=_h(n=32, stride=32 * 128 + 4)) == INVALID      # rows off the 16-byte boundary
    assert call(q=_h(n=32, stride=32 * 128 + 4, dtype=2), qo=_h(FAKE + 2, 32)) == INVALID
    assert call(qo=_h(FAKE + (1 << 30), n=16)) == INVALID        # another number of heads
    assert call(qo=_h(FAKE, n=32, dtype=2)) == INVALID           # in place in another type
    assert call(k=_h(n=8)) == INVALID                            # keys in, none out
    assert call(ko=_h(n=8)) == INVALID
    assert call(k=_h(n=8, dtype=1), ko=_h(n=8, dtype=1)) == INVALID  # another type than q's
    assert call(pos=None) == INVALID and call(pos=FAKE + 2) == INVALID
    assert call(rope=_rope(rot=24)) == UNSUPPORTED
    assert call(rope=_rope(rot=144)) == INVALID and call(rope=_rope(rot=0)) == INVALID
    assert call(rope=_rope(inter=2)) == INVALID and call(rope=_rope(freqs=None)) == INVALID
    assert call(rope=_rope(m=math.inf)) == INVALID and call(rope=_rope(reserved=1)) == INVALID
    assert call(qw=FAKE + 4) == INVALID
    assert call(qw=FAKE, eps=-1.0) == INVALID and call(kw=FAKE, eps=math.nan) == INVALID


def _c(dtype=kvd.F16, B=2, Hkv=8, D=128, pages=64, ps=64, cols=32, length=1000, **kw):
    s = kvd.PagedCacheStruct(dtype, B, Hkv, D, pages, ps, cols, length, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE,
                         None)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


BAD_CACHES = [
    (dict(dtype=7), INVALID), (dict(dtype=kvd.Q8_0), UNSUPPORTED), (dict(dtype=kvd.Q4_0), UNSUPPORTED),
    (dict(B=0), INVALID), (dict(Hkv=0), INVALID), (dict(pages=0), INVALID), (dict(cols=0), INVALID),
    (dict(D=96), UNSUPPORTED), (dict(D=256), UNSUPPORTED), (dict(ps=0), INVALID),
    (dict(ps=8), UNSUPPORTED), (dict(ps=72), UNSUPPORTED), (dict(length=-1), INVALID),
    (dict(length=64 * 32 + 1), INVALID), (dict(k=FAKE + 8), INVALID), (dict(v=None), INVALID),
    (dict(dtype=kvd.INT8, k_scale=None), INVALID), (dict(dtype=kvd.INT8, v_scale=FAKE + 4), INVALID),
    (dict(page_table=None), INVALID), (dict(page_table=FAKE + 2), INVALID), (dict(seq_lens=None), INVALID),
    (dict(dev_status=FAKE + 1), INVALID), (dict(pages=1 << 22), UNSUPPORTED),
]


def test_paged_refusals():
    L = kvd.lib()

    def append(c=None, k=None, v=None, n=4, starts=FAKE, rope=None, q=None, qo=None, D=128):
        return L.kvd_paged_append(C.byref(c or _c()), k or _h(D=D), v or _h(D=D), n, starts, rope, None, q,
                                  qo, None, 1e-6, None)

    def need(c=None, H=32, n=4, new=4):
        return L.kvd_paged_workspace_bytes(C.byref(c or _c()), H, n, new)

    def attn(c=None, q=None, n=4, starts=FAKE, new=4, scale=0.1, window=0, out=None, ws=FAKE, nb=None):
        return L.kvd_paged_attn(C.byref(c or _c()), q or _h(n=32), n, starts, new, scale, window,
                                out or _h(FAKE + (1 << 30), n=32), ws, need() if nb is None else nb, None)

    for kw, status in BAD_CACHES:
        c = _c(**kw)
        assert append(c) == status, kw
        assert attn(c) == status, kw
        assert need(c) == 0, kw
    assert append(n=0) == OK and attn(n=0) == OK and attn(new=0) == OK
    assert append(n=-1) == INVALID and attn(n=-1) == INVALID and attn(new=-1) == INVALID
    assert append(k=_h(n=4)) == INVALID and append(v=_h(n=16)) == INVALID
    assert append(v=_h(dtype=1)) == INVALID
    assert append(starts=None) == INVALID and attn(starts=FAKE + 2) == INVALID
    assert append(q=_h(n=32)) == INVALID and append(qo=_h(n=32)) == INVALID
    assert append(rope=_rope(rot=144)) == INVALID and append(rope=_rope(rot=40)) == UNSUPPORTED
    assert attn(q=_h(n=30)) == INVALID
    assert attn(q=_h(n=136), out=_h(FAKE + (1 << 30), n=136)) == UNSUPPORTED   # 17 heads a KV head
    assert attn(q=_h(n=32, dtype=1), out=_h(FAKE + (1 << 30), n=32, dtype=1)) == INVALID
    assert attn(q=_h(n=32, dtype=2), out=_h(FAKE + (1 << 30), n=32, dtype=2)) == INVALID
    assert attn(c=_c(kvd.INT8), q=_h(n=32, dtype=1)) == INVALID                # out of another type
    assert attn(out=_h(FAKE, n=32)) == INVALID                                 # in place
    assert attn(window=-1) == INVALID
    for scale in (0.0, -1.0, math.nan, math.inf):
        assert attn(scale=scale) == INVALID
    assert attn(ws=None) == WORKSPACE and attn(ws=FAKE + 64) == WORKSPACE
    assert attn(nb=need() - 1) == WORKSPACE
    assert need(H=30) == 0 and need(H=136) == 0 and need(n=0) == 0 and need(new=0) == 0


def test_binding_checks_shapes_before_the_library():
    t = {"k": torch.zeros(4, 2, 16, 64, dtype=torch.float16)}
    with pytest.raises(ValueError):          # not on a GPU
        kvd.PagedKVCache(kvd.F16, 1, 4, 2, 16, 4, head_dim=64, device="cpu")
    with pytest.raises(ValueError):          # pages of another type than the cache's
        kvd.PagedKVCache(kvd.BF16, 1, 4, 2, 16, 4, head_dim=64, device="cpu", tensors=t)
    with pytest.raises(ValueError):          # channels not dense
        kvd._heads(torch.zeros(3, 4, 128, dtype=torch.float16)[..., ::2])
    with pytest.raises(ValueError):          # heads not dense
        kvd._heads(torch.zeros(3, 8, 64, dtype=torch.float16)[:, ::2])
    with pytest.raises(ValueError):
        kvd._heads(torch.zeros(3, 8, 64, dtype=torch.float64))
    s = kvd._heads(torch.zeros(3, 12, 64, dtype=torch.bfloat16)[:, 4:8])
    assert (s.stride, s.dtype, s.n_heads) == (768, 1, 4)


def test_caches_too_long_to_count():
    """Lengths above 2^30 and more than 2^31 - 1 key tiles are refused, by every call."""
    L = kvd.lib()
    for kw in (dict(ps=1 << 16, cols=1 << 15, pages=4, length=(1 << 30) + 1),
               dict(ps=1 << 16, cols=1 << 15, pages=4, B=1 << 12, length=1 << 30)):
        c, k = C.byref(_c(**kw)), _h()
        assert L.kvd_paged_append(c, k, k, 4, FAKE, None, None, None, None, None, 1e-6, None) == UNSUPPORTED
        assert L.kvd_paged_attn(c, _h(n=32), 4, FAKE, 4, 0.1, 0, _h(FAKE + (1 << 30), n=32), FAKE, 1 << 40,
                                None) == UNSUPPORTED
        assert L.kvd_paged_workspace_bytes(c, 32, 4, 4) == 0
