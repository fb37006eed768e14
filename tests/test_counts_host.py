"""The bounds of count_ref.py: one key lost or taken twice falls outside of them, wherever it lies, and so do a
row whose weight a key does not get and a tile that the sums of a row leave out.  No GPU."""
import pytest
import torch

import count_ref as N
import long_context_decode_kv_gb300 as kvd

BF16, F16 = torch.bfloat16, torch.float16


def _cases():
    for dtype in (kvd.F16, kvd.BF16):
        for i, (rank, P, _, H, window, new, lens) in enumerate(N.LATENT):
            yield f"latent-{i}-{dtype}", dtype, rank, P, H, window, new, lens
        for i, (D, _, H, Hkv, window, new, parts) in enumerate(N.HEADS):
            yield f"heads-{i}-{dtype}", dtype, D, D, H // Hkv, window, new, N.lengths(dtype, D, new, parts)


@pytest.mark.parametrize("dtype,R,W,G,window,new,lens", [c[1:] for c in _cases()], ids=[c[0] for c in _cases()])
def test_a_key_more_or_less_is_out_of_bounds(dtype, R, W, G, window, new, lens):
    x = BF16 if dtype == kvd.BF16 else F16
    for b, (n, L) in enumerate(zip(new, lens)):
        if n == 0:
            continue
        rows, n, code = n * G, min(n, 3), N.codes(L, W, b, "cpu")     # (the last three tokens')
        for flat in (True, False):
            pick = N.picked(n, min(G, 2), W, flat)
            good = N.reference(code, pick, R, n, window, x)
            if flat:                                      # a row's weight stands out among all of them
                some = torch.isfinite(good["least"])
                more = (rows / 8 + 64) / (pick.numel() / 8 + 64) * rows / pick.numel()
                assert torch.all((2 * good["mass"][1] * more < good["least"])[some]), L
            lo = max(L - n - window + 1, 0) if window else 0
            if not flat or L - n - lo < 2:
                continue
            for t in {lo, lo + 1, (lo + L) // 2, (lo + L) // 2 // 64 * 64, L - n - 1, L - n}:
                if t < lo or t > L - n:
                    continue
                for kw in (dict(lost=t), dict(twice=t)):
                    bad = N.reference(code, pick, R, n, window, x, **kw)
                    assert N.apart(good["out"], bad["out"]).any(), (L, kw)
            if L - lo > 256:
                tile = torch.arange(lo // 64 * 64 + 64, lo // 64 * 64 + 128)
                bad = N.reference(code, pick, R, n, window, x, lost=tile)
                assert N.apart(good["lse"], bad["lse"]).any()
