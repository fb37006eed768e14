"""Attention, its statistics and accumulated weights over caches that tell every key and row apart
(count_ref.py): a key lost or counted twice where CTAs, tiles or pages meet is out of bounds."""
import math

import pytest
import torch

import count_ref as N
import latent_ref as LR
import long_context_decode_kv_gb300 as kvd
import paged_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
X = {kvd.F16: torch.float16, kvd.BF16: torch.bfloat16, kvd.INT8: torch.float16}


def _check(c, z, q, pick, new, window):
    """c: the cache, z[b][g]: the codes, q and pick: the rows' queries."""
    latent = isinstance(c, kvd.LatentCache)
    Hkv = LR.heads_of(c)
    T, H, _ = q.shape
    G, V = H // Hkv, c.rank if latent else c.head_dim
    starts = torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int32, device=DEV)
    out = torch.full((T, H, V), math.nan, device=DEV, dtype=q.dtype)
    lse = torch.full((T, H), math.nan, device=DEV)
    ws = (kvd.make_latent_workspace if latent else kvd.make_paged_workspace)(c, H, T, max(new))
    (kvd.latent_attn if latent else kvd.paged_attn)(c, q, starts, max(new), 1.0, out, ws, window=window, lse=lse)
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    mass = torch.rand(c.batch, Hkv, c.len, generator=g, device=DEV) * 1e-3
    got = mass.clone()
    kvd.paged_mass(c, q, lse, starts, max(new), 1.0, got, decay=0.75, window=window)
    assert c.device_status() == 0
    for b, n in enumerate(new):
        L, s = int(c.seq_lens[b]), int(starts[b])
        for h in range(Hkv):
            want = N.reference(z[b][h], pick[s:s + n, h * G:h * G + G], V, n, window, q.dtype, mass[b, h, :L], 0.75)
            what = f"sequence {b}, head {h}: "
            LR.assert_close(out[s:s + n, h * G:h * G + G], want["out"], what + "out")
            LR.assert_close(lse[s:s + n, h * G:h * G + G], want["lse"], what + "lse")
            LR.assert_close(got[b, h, :L], want["mass"], what + "mass")
            assert torch.equal(got[b, h, L:], mass[b, h, L:])


@pytest.mark.parametrize("dtype", [kvd.F16, kvd.BF16])
@pytest.mark.parametrize("flat", [True, False])
@pytest.mark.parametrize("rank,P,page,H,window,new,lens", N.LATENT)
def test_latent(dtype, flat, rank, P, page, H, window, new, lens):
    cols = max((n + page - 1) // page for n in lens) + 1
    c, z = N.latent(dtype, lens, page, rank, P, 3, DEV, R.scattered_tables(len(lens), cols, 7, "cpu"))
    pick = N.picked(sum(new), H, P, flat)
    _check(c, [[x] for x in z], N.queries(pick, rank + P, rank, X[dtype], DEV), pick, new, window)


@pytest.mark.parametrize("dtype", [kvd.F16, kvd.BF16, kvd.INT8])
@pytest.mark.parametrize("flat", [True, False])
@pytest.mark.parametrize("D,page,H,Hkv,window,new,parts", N.HEADS)
def test_heads(dtype, flat, D, page, H, Hkv, window, new, parts):
    lens = N.lengths(dtype, D, new, parts)
    cols = max((n + page - 1) // page for n in lens) + 1
    c, z = N.heads(dtype, lens, Hkv, D, page, 3, DEV, R.scattered_tables(len(lens), cols, 7, "cpu"))
    pick = N.picked(sum(new), H, D, flat)
    _check(c, z, N.queries(pick, D, 0, X[dtype], DEV), pick, new, window)
