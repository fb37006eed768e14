"""64-bit references of the latent cache's calls, the accumulated weights and the eviction, and the
bounds their tests use.

Bounds count half steps u = finfo(type).eps / 2 of each rounding and the f32 arithmetic between them:
  logit      z of W channels: the products are exact in f32, their sum and the scale are off by at most
             2 W steps of 2^-23 of the sum of |products| (dz)
  weight     exp of it: dz, and 2^-22 of the exponential itself
  sums       over N keys or rows in chains of N / 8 + 64 additions at most
  output     weights rounded to the row's type (u_p), in f16 not below 2^-31 of the largest; the f32
             accumulation; the output's rounding
  lse        dz, the sum's steps, and 8 roundings of its size
"""
import math

import torch

import long_context_decode_kv_gb300 as kvd
from paged_ref import rounding, rows_of, u


def sides(cache, b, g, total):
    """Keys and values [total, ..] of sequence b and KV head g, in float64."""
    if isinstance(cache, kvd.LatentCache):
        ids = cache.page_table[b, :(total + cache.page_size - 1) // cache.page_size].long()
        x = cache.rows[ids].flatten(0, 1)[:total].double()
        return x, x[:, :cache.rank]
    out = []
    for n in "kv":
        x = rows_of(cache.t[n], cache.page_table[b], total, g).double()
        if cache.dtype == kvd.INT8:
            x = x * rows_of(cache.t[n + "_scale"], cache.page_table[b], total, g).double()[:, None]
        out.append(x)
    return out


def heads_of(cache):
    return 1 if isinstance(cache, kvd.LatentCache) else cache.n_kv_heads


def attn(cache, q, starts, lens, scale, window=0, decay=1.0, mass=None):
    """A dict of (value, bound) in float64: out, lse, and with a mass the accumulated weights.
    Rows of no sequence are NaN, and so are weights at or behind a sequence's length."""
    T, H, W = q.shape
    Hkv = heads_of(cache)
    G = H // Hkv
    V = cache.rank if isinstance(cache, kvd.LatentCache) else W
    f64 = dict(dtype=torch.float64, device=q.device)
    out, tol = torch.full((T, H, V), math.nan, **f64), torch.zeros(T, H, V, **f64)
    lse, lse_tol = torch.full((T, H), math.nan, **f64), torch.zeros(T, H, **f64)
    got = {"out": (out, tol), "lse": (lse, lse_tol)}
    if mass is not None:
        add, add_tol = torch.full(mass.shape, math.nan, **f64), torch.zeros(mass.shape, **f64)
        got["mass"] = (add, add_tol)
    up = u(q.dtype)
    for b in range(cache.batch):
        s0, s1, L = int(starts[b]), int(starts[b + 1]), int(lens[b])
        n = s1 - s0
        t = torch.arange(L, device=q.device)
        p = torch.arange(L - n, L, device=q.device)
        seen = t <= p[:, None]
        if window:
            seen &= t > p[:, None] - window
        for g in range(Hkv):
            k, v = sides(cache, b, g, L)
            if mass is not None:
                add[b, g, :L] = 0.0
                if decay:
                    add[b, g, :L - n] = mass[b, g, :L - n].double() * decay
                add_tol[b, g, :L] = add[b, g, :L].abs() * 2.0 ** -23
            if n == 0:
                continue
            for h in range(g * G, g * G + G):
                qq = q[s0:s1, h].double()
                z = torch.where(seen, qq @ k.T * scale, -math.inf)
                mag = torch.where(seen, qq.abs() @ k.abs().T * scale, 0.0)
                dz = 2 * W * 2.0 ** -23 * mag.amax(-1, keepdim=True)
                top = z.amax(-1, keepdim=True).clamp_min(-1e300)
                e = (z - top).exp()
                l = e.sum(-1, keepdim=True)
                w = e / l.clamp_min(1e-300)
                a = w @ v.abs()
                N = seen.sum(-1, keepdim=True).double()
                steps = (N / 8 + 64) * 2.0 ** -23
                err = a * (up + dz + steps) * 1.01
                if q.dtype == torch.float16:
                    err = err + 2.0 ** -25 * (seen.double() @ v.abs()) / l.clamp_min(1e-300)
                out[s0:s1, h] = w @ v
                tol[s0:s1, h] = rounding(out[s0:s1, h], err, q.dtype)
                s = (top + l.clamp_min(1e-300).log()).squeeze(-1)
                lse[s0:s1, h] = torch.where(l.squeeze(-1) > 0, s, -math.inf)
                lse_err = (dz + steps).squeeze(-1) + 8 * 2.0 ** -24 * (s.abs() + top.squeeze(-1).abs() + 16)
                lse_tol[s0:s1, h] = torch.where(l.squeeze(-1) > 0, lse_err, 0.0)
                if mass is not None:
                    rel = dz + lse_err[:, None] + 2.0 ** -22
                    add[b, g, :L] += w.sum(0)
                    add_tol[b, g, :L] += (w * rel).sum(0) * 1.01
            if mass is not None:
                add_tol[b, g, :L] += add[b, g, :L].abs() * (n * G / 8 + 64) * 2.0 ** -23
    return got


def assert_close(got, want, what=""):
    """Against (value, bound); infinities have to agree, places without a value are skipped."""
    value, tol = want
    g = got.double()
    some = ~value.isnan()
    off = torch.where(value.isinf(), (g != value).double() * math.inf, (g - value).abs())
    off = torch.where(value.isinf() & (g == value), 0.0, off)
    bad = some & ~(off <= tol)
    if bad.any():
        i = tuple(int(x) for x in torch.nonzero(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds, first at {i}: "
                             f"got {float(g[i])}, want {float(value[i])} +- {float(tol[i])}")


def kept_of(mass, total, keep, sink, recent):
    """Indices that stay of one (sequence, head), ascending, by the definition."""
    if total <= keep:
        return list(range(total))
    m = [-math.inf if x != x else x for x in mass[:total].tolist()]
    nan = [x != x for x in mass[:total].tolist()]
    mid = sorted(range(sink, total - recent), key=lambda t: (nan[t], -m[t], t))
    return sorted(list(range(sink)) + mid[:keep - sink - recent] + list(range(total - recent, total)))
