"""64-bit references of the norm/rotation, the paged append and the paged attention,
and the bounds their tests use.

Bounds count half steps u = finfo(type).eps / 2 of each rounding and the f32 arithmetic
between them, element by element:
  rotation   angle: its fraction of a turn rounded to f32 (pi 2^-25), sine and cosine
             (2 units), the products and the sum (3 roundings): under 16 * 2^-24 of
             |u| + |v|.  Norm: a sum of D squares in chains of at most D/32 + 13 additions,
             half of it after the root, then root, quotient and two products.
  attention  weights rounded to the input type (u_p), each logit off by D steps of its
             sum of |products|, accumulation over N keys in steps of 16, and the output.
"""
import math

import torch

import long_context_decode_kv_gb300 as kvd


def u(dtype):
    return torch.finfo(dtype).eps / 2


def freqs(rot, base=10000.0, scaling="none", factor=1.0, orig=0.0, low=0.0, high=0.0):
    """(radians per position [rot / 2] float64, mscale), from the definitions."""
    out, m = [], 1.0
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    if scaling in ("yarn", "bands") and low == high == 0:
        low, high = 1.0, (32.0 if scaling == "yarn" else 4.0)
    if scaling == "yarn":
        m = 0.1 * math.log(factor) + 1
        at = [rot * math.log(orig / (t * 2 * math.pi)) / (2 * math.log(base)) for t in (high, low)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        keep = 1.0
        if scaling == "linear":
            keep = 0.0
        elif scaling == "yarn":
            keep = 1 - min(max((i - lo) / max(hi - lo, 0.001), 0), 1)
        elif scaling == "bands":
            keep = min(max((orig * f / (2 * math.pi) - low) / (high - low), 0), 1)
        out.append(f * keep + f / factor * (1 - keep))
    return torch.tensor(out, dtype=torch.float64), m


def turned(x, pos, f, m, interleaved, w=None, eps=1e-6):
    """(y, bound of |error| before the output's rounding) for x [T, h, D], in float64."""
    x = x.double()
    D = x.shape[-1]
    n_norm = 0
    if w is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
        n_norm = (D / 32 + 13) / 2 + 6
    y, mag = x.clone(), x.abs()
    if f is not None:
        r = 2 * f.numel()
        f = f.to(x.device)
        a = pos.double()[:, None, None] * f
        c, s = a.cos() * m, a.sin() * m
        i = torch.arange(r // 2, device=x.device)
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
        y[..., p] = x[..., p] * c - x[..., q] * s
        y[..., q] = x[..., q] * c + x[..., p] * s
        both = (x[..., p].abs() + x[..., q].abs()) * m
        mag = mag.clone()
        mag[..., p] = both
        mag[..., q] = both
    return y, mag * (16 + n_norm) * 2.0 ** -24


def rounding(y, err, dtype):
    """Bound of |error| once y with that error is rounded to dtype."""
    return err + u(dtype) * (y.abs() + err) * (1 + 2.0 ** -20) + torch.finfo(dtype).smallest_normal * u(dtype)


def scattered_tables(B, cols, seed, device):
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(B * cols, generator=g).view(B, cols).int().to(device)


def rows_of(pages, table_row, total, head):
    """Tokens [0, total) of one sequence and KV head: pages [n, Hkv, ps, ...]."""
    ps = pages.shape[2]
    ids = table_row[:(total + ps - 1) // ps].long()
    x = pages[ids, head]
    return x.reshape(-1, *x.shape[2:])[:total]


def attn_ref(cache, q, starts, lens, scale, window=0):
    """(out, bound) in float64 for paged_attn; rows behind the last sequence are None-valued (NaN)."""
    T, H, D = q.shape
    G = H // cache.n_kv_heads
    out = torch.full(q.shape, math.nan, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    up = u(q.dtype)
    for b in range(cache.batch):
        s0, s1, L = int(starts[b]), int(starts[b + 1]), int(lens[b])
        n = s1 - s0
        if n == 0:
            continue
        p = torch.arange(L - n, L, device=q.device)
        t = torch.arange(L, device=q.device)
        seen = t <= p[:, None]
        if window:
            seen &= t > p[:, None] - window
        for g in range(cache.n_kv_heads):
            k = rows_of(cache.k, cache.page_table[b], L, g).double()
            v = rows_of(cache.v, cache.page_table[b], L, g).double()
            big = 0.0
            if cache.dtype == kvd.INT8:
                k = k * rows_of(cache.k_scale, cache.page_table[b], L, g).double()[:, None]
                vs = rows_of(cache.v_scale, cache.page_table[b], L, g).double()
                v = v * vs[:, None]
                big = float(vs.max()) * 127 if L else 0.0
            for h in range(g * G, g * G + G):
                qq = q[s0:s1, h].double()
                z = torch.where(seen, qq @ k.T * scale, -math.inf)
                mag = torch.where(seen, qq.abs() @ k.abs().T * scale, 0.0).amax(-1, keepdim=True)
                top = z.amax(-1, keepdim=True).clamp_min(-1e300)
                e = (z - top).exp()
                l = e.sum(-1, keepdim=True).clamp_min(1e-300)
                w = e / l
                o = w @ v
                a = w @ v.abs()
                N = seen.sum(-1, keepdim=True).double()
                # f16 weights below 2^-14 of the largest keep 2^-25 of it
                small = 2.0 ** -25 * (seen.double() @ v.abs()) / l + 2.0 ** -23 * big * N / l
                err = a * (up + 2 * D * 2.0 ** -23 * mag + (N / 8 + 64) * 2.0 ** -23) * 1.01
                if q.dtype == torch.float16:
                    err = err + small
                out[s0:s1, h] = o
                tol[s0:s1, h] = rounding(o, err, q.dtype)
    return out, tol


def assert_within(got, want, tol, what=""):
    off = (got.double() - want).abs()
    bad = ~(off <= tol)
    if bad.any():
        i = tuple(int(x) for x in torch.nonzero(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds, first at {i}: "
                             f"got {float(got[i])}, want {float(want[i])} +- {float(tol[i])}")
