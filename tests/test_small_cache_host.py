"""Host side of the latent cache's calls, the accumulated weights and the eviction: refusals, and the
binding's checks.  No GPU."""
import ctypes as C
import math

import pytest
import torch

import latent_ref as LR
import long_context_decode_kv_gb300 as kvd
from test_paged_host import BAD_CACHES, FAKE, INVALID, OK, UNSUPPORTED, WORKSPACE, _c, _h, _rope

FAR = FAKE + (1 << 30)


@pytest.fixture(scope="module", autouse=True)
def _built():
    from long_context_decode_kv_gb300 import build
    build.build()


def _l(dtype=kvd.BF16, B=2, rank=512, P=64, pages=64, ps=64, cols=32, length=1000, **kw):
    s = kvd.LatentCacheStruct(dtype, B, rank, P, pages, ps, cols, length, FAKE, FAKE, FAKE, None)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def _p(x=FAKE, n=16, stride=16 * 192, head=192, dtype=1):
    return kvd.PartsStruct(x, stride, head, dtype, n)


BAD_LATENT = [
    (dict(dtype=7), INVALID), (dict(dtype=kvd.INT8), UNSUPPORTED), (dict(dtype=kvd.Q8_0), UNSUPPORTED),
    (dict(B=0), INVALID), (dict(rank=0), INVALID), (dict(rank=64), UNSUPPORTED), (dict(rank=640), UNSUPPORTED),
    (dict(rank=200), UNSUPPORTED), (dict(P=0), INVALID), (dict(P=8), UNSUPPORTED), (dict(P=80), UNSUPPORTED),
    (dict(pages=0), INVALID), (dict(cols=0), INVALID), (dict(ps=0), INVALID), (dict(ps=24), UNSUPPORTED),
    (dict(length=-1), INVALID), (dict(length=64 * 32 + 1), INVALID), (dict(rows=None), INVALID),
    (dict(rows=FAKE + 8), INVALID), (dict(page_table=None), INVALID), (dict(seq_lens=FAKE + 2), INVALID),
    (dict(dev_status=FAKE + 1), INVALID), (dict(pages=1 << 26), UNSUPPORTED),
    (dict(ps=1 << 16, cols=1 << 15, pages=4, length=(1 << 30) + 1), UNSUPPORTED),
]


def _append(c=None, lat=None, k=None, n=4, starts=FAKE, rope=None, w=None, q=None, qo=None, eps=1e-6):
    return kvd.lib().kvd_latent_append(C.byref(c or _l()), lat or _h(n=1, D=512, dtype=1),
                                       k or _h(n=1, D=64, dtype=1), n, starts, rope, w, q, qo, eps, None)


def _need(c=None, H=16, n=4, new=4):
    return kvd.lib().kvd_latent_workspace_bytes(C.byref(c or _l()), H, n, new)


def _attn(c=None, q=None, n=4, starts=FAKE, new=4, scale=0.1, window=0, out=None, lse=None, ws=FAKE, nb=None):
    return kvd.lib().kvd_latent_attn(C.byref(c or _l()), q or _h(n=16, D=576, dtype=1), n, starts, new, scale,
                                     window, out or _h(FAR, n=16, D=512, dtype=1), lse, ws,
                                     (_need() or 1 << 40) if nb is None else nb, None)


def _mass(c=None, q=None, lse=FAKE, n=4, starts=FAKE, new=4, scale=0.1, window=0, mass=FAKE, stride=2048,
          decay=1.0, out=FAR, out_stride=2048):
    latent = c is None or isinstance(c, kvd.LatentCacheStruct)
    f = kvd.lib().kvd_latent_mass if latent else kvd.lib().kvd_paged_mass
    q = q or (_h(n=16, D=576, dtype=1) if latent else _h(n=32))
    return f(C.byref(c or _l()), q, lse, n, starts, new, scale, window, mass, stride, decay, out, out_stride, None)


def _evict(c=None, mass=FAKE, stride=2048, keep=256, sink=4, recent=32, to=FAKE, cols=8, kept=FAKE,
           lens=FAKE + 64, mass_out=FAR, out_stride=256):
    f = kvd.lib().kvd_latent_evict if c is None or isinstance(c, kvd.LatentCacheStruct) else \
        kvd.lib().kvd_paged_evict
    return f(C.byref(c or _l()), mass, stride, keep, sink, recent, to, cols, kept, lens, mass_out, out_stride, None)


def test_bad_caches_are_refused_by_every_call():
    for kw, status in BAD_LATENT:
        c = _l(**kw)
        assert _append(c) == status, kw
        assert _attn(c, nb=1 << 40) == status, kw
        assert _mass(c) == status, kw
        assert _evict(c) == status, kw
        assert _need(c) == 0, kw
    for kw, status in BAD_CACHES:
        c = _c(**kw)
        assert _mass(c) == status, kw
        assert _evict(c) == status, kw


def test_append_refusals():
    assert _append(n=0) == OK and _append(n=-1) == INVALID
    assert _append(lat=_h(n=1, D=512, dtype=3)) == INVALID
    assert _append(lat=_h(FAKE + 2, n=1, D=512, dtype=1)) == INVALID
    assert _append(lat=_h(n=2, D=512, dtype=1)) == INVALID                    # one head
    assert _append(lat=_h(n=1, D=512, dtype=1, stride=504)) == INVALID        # tokens overlap
    assert _append(k=_h(n=1, D=64, dtype=1, stride=68)) == INVALID            # rows off the 16-byte boundary
    assert _append(k=_h(n=1, D=64, dtype=0)) == INVALID                       # another type than c's
    assert _append(starts=None) == INVALID and _append(starts=FAKE + 2) == INVALID
    assert _append(w=FAKE + 4) == INVALID and _append(w=FAKE, eps=-1.0) == INVALID
    assert _append(w=FAKE, eps=math.nan) == INVALID
    assert _append(rope=_rope(rot=80)) == INVALID and _append(rope=_rope(rot=24)) == UNSUPPORTED
    assert _append(rope=_rope(inter=2)) == INVALID
    assert _append(q=_p()) == INVALID and _append(qo=_p()) == INVALID         # one without the other
    far = _p(FAR, head=576, stride=16 * 576)
    for q in (_p(FAKE + 8), _p(None), _p(n=0), _p(dtype=0), _p(head=56), _p(head=196), _p(stride=16 * 192 + 4),
              _p(stride=15 * 192 + 32), _p(n=8), _p(head=-192), _p(head=1 << 41)):
        assert _append(q=q, qo=far) == INVALID
    assert _append(q=_p(), qo=_p(FAR, head=32)) == INVALID
    assert _append(q=_p(), qo=_p(FAKE, head=576, stride=16 * 576)) == INVALID  # in place in another layout


def test_attention_refusals():
    assert _attn(n=0) == OK and _attn(new=0) == OK
    assert _attn(n=-1) == INVALID and _attn(new=-1) == INVALID and _attn(window=-1) == INVALID
    assert _attn(q=_h(n=16, D=576, dtype=0), out=_h(FAR, n=16, D=512, dtype=0)) == INVALID   # the cache is bf16
    assert _attn(q=_h(n=16, D=576, dtype=2), out=_h(FAR, n=16, D=512, dtype=2)) == INVALID
    assert _attn(out=_h(FAR, n=16, D=512, dtype=0)) == INVALID
    assert _attn(out=_h(FAR, n=8, D=512, dtype=1)) == INVALID
    assert _attn(out=_h(FAKE, n=16, D=512, dtype=1)) == INVALID                              # in place
    assert _attn(q=_h(n=16, D=512, dtype=1)) == INVALID                                      # stride below a token
    assert _attn(q=_h(n=1025, D=576, dtype=1), out=_h(FAR, n=1025, D=512, dtype=1), nb=1 << 40) == UNSUPPORTED
    for scale in (0.0, -1.0, math.nan, math.inf):
        assert _attn(scale=scale) == INVALID
    assert _attn(starts=None) == INVALID and _attn(starts=FAKE + 2) == INVALID
    assert _attn(lse=FAKE + 4) == INVALID
    assert _attn(ws=None) == WORKSPACE and _attn(ws=FAKE + 64) == WORKSPACE and _attn(nb=0) == WORKSPACE
    assert _need(H=0) == 0 and _need(H=1025) == 0 and _need(n=0) == 0 and _need(new=0) == 0


def test_paged_lse_refusals():
    f = kvd.lib().kvd_paged_attn_lse
    for lse in (None, FAKE + 4):
        assert f(C.byref(_c()), _h(n=32), 4, FAKE, 4, 0.1, 0, _h(FAR, n=32), lse, FAKE, 1 << 40, None) == INVALID
    assert f(C.byref(_c()), _h(n=32), 0, FAKE, 4, 0.1, 0, _h(FAR, n=32), FAKE, FAKE, 1 << 40, None) == OK
    assert f(C.byref(_c()), _h(n=32), 4, FAKE, 4, 0.1, 0, _h(FAR, n=32), FAKE, None, 0, None) == WORKSPACE


def test_a_call_without_rows_is_a_no_op_with_statistics_too():
    """An empty tensor's pointer is NULL: without rows no call asks for q, out, lse or a workspace."""
    f, lse = kvd.lib().kvd_paged_attn, kvd.lib().kvd_paged_attn_lse
    for n, new in ((0, 4), (4, 0), (0, 0)):
        assert f(C.byref(_c()), None, n, None, new, 0.1, 0, None, None, 0, None) == OK
        assert lse(C.byref(_c()), None, n, None, new, 0.1, 0, None, None, None, 0, None) == OK
        assert kvd.lib().kvd_latent_attn(C.byref(_l()), None, n, None, new, 0.1, 0, None, None, None, 0, None) == OK
    for n, new in ((0, -1), (-1, 0)):
        assert lse(C.byref(_c()), None, n, None, new, 0.1, 0, None, None, None, 0, None) == INVALID
    assert lse(C.byref(_c(B=0)), None, 0, None, 0, 0.1, 0, None, None, None, 0, None) == INVALID


def test_mass_refusals():
    for c in (_l(), _c()):
        assert _mass(c, n=-1) == INVALID and _mass(c, new=-1) == INVALID and _mass(c, window=-1) == INVALID
        for decay in (-0.5, math.nan, math.inf):
            assert _mass(c, decay=decay) == INVALID
        assert _mass(c, mass=None) == INVALID and _mass(c, mass=FAKE + 2) == INVALID
        assert _mass(c, stride=999) == INVALID and _mass(c, out_stride=999) == INVALID       # below len
        assert _mass(c, out=None) == INVALID and _mass(c, out=FAR + 1) == INVALID
        assert _mass(c, out=FAKE, out_stride=1024) == INVALID                                 # in place, other rows
        assert _mass(c, lse=None) == INVALID and _mass(c, lse=FAKE + 4) == INVALID
        assert _mass(c, starts=None) == INVALID
        for scale in (0.0, -1.0, math.nan, math.inf):
            assert _mass(c, scale=scale) == INVALID
    assert _mass(_c(), q=_h(n=30)) == INVALID and _mass(_c(), q=_h(n=136)) == UNSUPPORTED
    assert _mass(_c(), q=_h(n=32, dtype=1)) == INVALID and _mass(_c(), q=_h(n=32, dtype=2)) == INVALID
    assert _mass(_l(), q=_h(n=16, D=576, dtype=0)) == INVALID
    assert _mass(_l(), q=_h(n=1025, D=576, dtype=1)) == UNSUPPORTED


def test_evict_refusals():
    for c in (_l(), _c()):
        assert _evict(c, keep=0) == INVALID and _evict(c, sink=-1) == INVALID and _evict(c, recent=-1) == INVALID
        assert _evict(c, sink=200, recent=57) == INVALID                      # above keep
        assert _evict(c, keep=(1 << 31) - 1, sink=(1 << 31) - 1, recent=1, out_stride=1 << 31) == INVALID
        assert _evict(c, mass=None) == INVALID and _evict(c, stride=999) == INVALID
        assert _evict(c, to=None) == INVALID and _evict(c, to=FAKE + 2) == INVALID
        assert _evict(c, cols=3) == INVALID and _evict(c, cols=0) == INVALID   # 192 rows for 256
        assert _evict(c, kept=None) == INVALID and _evict(c, lens=None) == INVALID
        assert _evict(c, lens=FAKE) == INVALID                                 # seq_lens itself
        assert _evict(c, out_stride=255) == INVALID and _evict(c, mass_out=FAKE) == INVALID
        assert _evict(c, mass_out=FAR + 2) == INVALID


def test_workspace_grows_with_the_rows():
    f = kvd.lib().kvd_latent_workspace_bytes
    sizes = [f(C.byref(_l()), 16, 4, n) for n in (1, 2, 4, 100)]
    assert sizes == sorted(sizes) and sizes[0] > 0 and all(s % 256 == 0 for s in sizes)
    assert f(C.byref(_l(rank=128)), 16, 4, 4) < sizes[2]


def test_binding_checks_shapes_before_the_library():
    with pytest.raises(ValueError):          # not on a GPU
        kvd.LatentCache(kvd.BF16, 1, 4, 16, 4, device="cpu")
    with pytest.raises(kvd.KvdError):
        kvd.LatentCache(kvd.INT8, 1, 4, 16, 4, device="cpu")
    with pytest.raises(ValueError):          # pages of another type than the cache's
        kvd.LatentCache(kvd.BF16, 1, 4, 16, 4, device="cpu", tensors={"rows": torch.zeros(4, 16, 576)})
    m = torch.zeros(3, 2, 40)
    assert kvd._mass(m, 3, 2, 40, "m") == (m.data_ptr(), 40)
    assert kvd._mass(m[:, :, 4:], 3, 2, 30, "m")[1] == 40
    assert kvd._mass(None, 3, 2, 40, "m") == (None, 0)
    for bad, least in ((m, 41), (m.half(), 10), (m[:, ::2], 10), (m[:2], 10), (m[:, :, ::2], 10),
                       (torch.zeros(3, 3, 40)[:, :2], 10)):
        with pytest.raises(ValueError):
            kvd._mass(bad, 3, 2, least, "m")
    n, h, s0, s1 = kvd._part_strides(torch.zeros(5, 4, 192)[:, :, 128:], "q")
    assert (n, h, s0, s1) == (5, 4, 768, 192)
    with pytest.raises(ValueError):
        kvd._part_strides(torch.zeros(5, 4, 192)[:, :, ::2], "q")
    with pytest.raises(ValueError):
        kvd._lse(torch.zeros(3, 4), 3, 5)


def test_the_reference_of_the_eviction():
    """What the GPU tests hold the call to, on a case worked by hand."""
    m = torch.tensor([9.0, 1.0, 5.0, math.nan, 5.0, -0.0, 0.0, 7.0, 2.0])
    assert LR.kept_of(m, 9, 9, 0, 0) == list(range(9))
    assert LR.kept_of(m, 9, 4, 1, 1) == [0, 2, 7, 8]         # 7, and of the two 5s the lower index
    assert LR.kept_of(m, 9, 8, 0, 0) == [0, 1, 2, 4, 5, 6, 7, 8]
    assert LR.kept_of(m, 8, 7, 0, 1) == [0, 1, 2, 4, 5, 6, 7]
    assert LR.kept_of(m, 8, 5, 0, 1) == [0, 1, 2, 4, 7]
