"""Caches whose results tell every single key and row apart, with their values and bounds in float64.

Keys hold whole numbers and a query picks one of them, so a logit is a small whole number and exact in f32
(the scale is 1); value row t is the unit vector of channel t % R, so that output channel c is the share of
the keys t = c, c + R, ..: one key lost or taken twice moves it by one part in their number.  Bounds, from
half steps u = finfo(type).eps / 2:
  weight    base-2 exponent of at most z2 + 16 places: 4 roundings of it, and 2^-22 of each of 5 exponentials
            (itself, the reference's two moves, a join's factor, and one to spare)
  sums      chains of N / 8 + 64 additions, 2^-23 each
  output    weights rounded to the row's type twice u_p apart, f16 not below 2^-31 (int8 2^-24) of the largest
  lse       the sums' steps, the logarithm (2 units of a number below 32: 2^-18), 4 roundings of its size
"""
import math

import torch

import long_context_decode_kv_gb300 as kvd

LEVELS = 4  # logits 0 .. 3


def codes(n, W, seed, device):
    """Whole numbers [n, W] in [0, LEVELS)."""
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, LEVELS, (n, W), generator=g).to(device)


def picked(T, H, channels, flat):
    """The channel that each row's query picks [T, H] (-1: none, all logits are 0)."""
    if flat:
        return torch.full((T, H), -1)
    return (torch.arange(T)[:, None] * 5 + torch.arange(H) * 3) % channels


def reference(code, pick, R, n, window, dtype, mass=None, decay=1.0, lost=None, twice=None):
    """One sequence and KV head: the last n of the code's keys are the queries' tokens.  pick [n, G].
    Returns {name: (value, bound)} of out [n, G, R], lse [n, G] and the weights [L] (behind decay times a mass
    [L], if there is one), and "least": the least weight that a row gave each key.
    lost, twice: a key that the calculation leaves out, or counts twice (the bounds stay)."""
    L, dev = code.shape[0], code.device
    G = pick.shape[1]
    f64 = dict(dtype=torch.float64, device=dev)
    t = torch.arange(L, device=dev)
    p = torch.arange(L - n, L, device=dev)
    times = (t <= p[:, None]).double()
    if window:
        times *= t > p[:, None] - window
    N = times.sum(-1)
    if lost is not None:
        times[:, lost] = 0.0
    if twice is not None:
        times[:, twice] *= 2.0
    up = torch.finfo(dtype).eps / 2
    out, out_tol = torch.zeros(n, G, R, **f64), torch.zeros(n, G, R, **f64)
    lse, lse_tol = torch.zeros(n, G, **f64), torch.zeros(n, G, **f64)
    add, add_tol = torch.zeros(L, **f64), torch.zeros(L, **f64)
    least = torch.full((L,), math.inf, **f64)
    if mass is not None and decay:
        add[:L - n] = mass[:L - n].double() * decay
        add_tol = add * 2.0 ** -23
    for h in range(G if n else 0):
        z = torch.stack([torch.zeros(L, **f64) if c < 0 else code[:, c].double() for c in pick[:, h].tolist()])
        e = times * z.exp()
        l = e.sum(-1, keepdim=True)
        w = e / l
        z2 = LEVELS * math.log2(math.e)
        dw = (4 * (z2 + 16)) * 2.0 ** -24 + 5 * 2.0 ** -22
        steps = (N / 8 + 64)[:, None] * 2.0 ** -23
        y = torch.zeros(n, R, **f64).index_add_(1, t % R, w)
        seen = torch.zeros(n, R, **f64).index_add_(1, t % R, (times > 0).double())
        top = (times * z.exp()).amax(-1, keepdim=True)
        err = y * (up + dw + 2 * steps) + 2.0 ** -24 * seen * top / l
        out[:, h], out_tol[:, h] = y, err + up * (y + err) * (1 + 2.0 ** -20)
        s = l.squeeze(-1).log()
        lse[:, h] = s
        lse_tol[:, h] = steps.squeeze(-1) + dw + 2.0 ** -18 + 4 * 2.0 ** -24 * (s.abs() + 16)
        rel = dw + lse_tol[:, h, None] + 4 * 2.0 ** -24 * (s.abs()[:, None] + 16)
        add += w.sum(0)
        least = torch.minimum(least, torch.where(times > 0, w, math.inf).amin(0))
        add_tol += (w * rel).sum(0)
    add_tol = add_tol + add * (n * G / 8 + 64) * 2.0 ** -23
    return {"out": (out, out_tol), "lse": (lse, lse_tol), "mass": (add, add_tol), "least": least}


# (rank, rotated channels, page, heads, window, new tokens, lengths) of latent caches: single tokens whose keys are
# cut between CTAs, groups of heads, chunks, windows.  An output channel counts at most 31 keys, so that one more
# or less is over 3 % of it where bf16's roundings are 1.6 (twice two half steps of 2^-8).
LATENT = [
    (512, 64, 64, 40, 0, [1, 1, 1], [15001, 9, 8000]),
    (512, 64, 16, 130, 0, [1, 2], [9000, 300]),
    (512, 16, 128, 16, 4000, [1, 1], [15000, 64]),
    (384, 48, 48, 24, 0, [40, 0, 1], [900, 50, 11000]),
    (256, 32, 32, 12, 100, [70, 1, 33], [900, 7000, 33]),
    (256, 64, 64, 64, 0, [9, 1], [7500, 65]),
    (128, 16, 16, 7, 0, [100, 1], [3900, 3]),
]
# (channels, page, query heads, KV heads, window, new tokens, lengths in KV caches' channels: 30 bf16, 150 others)
HEADS = [
    (128, 64, 8, 2, 0, [1, 1, 1], [1.0, 0.01, 0.5]),
    (64, 16, 32, 2, 0, [1, 2], [1.0, 0.3]),
    (64, 64, 8, 8, 500, [3, 1], [1.0, 0.7]),
    (128, 48, 12, 2, 0, [40, 0, 1], [0.3, 0.1, 1.0]),
    (128, 128, 10, 2, 70, [129, 1], [0.4, 1.0]),
    (64, 32, 4, 1, 0, [200, 33], [0.5, 0.2]),
]


def lengths(dtype, D, new, parts):
    """The lengths of a line of HEADS: up to 30 keys a channel in bf16, up to 150 in f16 and int8."""
    most = (30 if dtype == kvd.BF16 else 150) * D
    return [max(int(most * x), n) for x, n in zip(parts, new)]


def apart(a, b):
    """Which places of b's values lie outside a's bounds by b's own bound or more."""
    return (a[0] - b[0]).abs() > a[1] + b[1]


def latent(dtype, lens, page, rank, P, seed, device, table):
    """A latent cache of such rows, the whole numbers in its rotated part; and the codes [L, P] of each."""
    B, cols = table.shape
    c = kvd.LatentCache(dtype, B, B * cols, page, cols, rank=rank, rope_dim=P, device=device)
    c.page_table.copy_(table)
    c.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
    c.len = max(lens)
    c.rows.fill_(math.nan)
    out = []
    for b, n in enumerate(lens):
        t = torch.arange(n, device=device)
        z = codes(n, P, seed + b, device)
        row = torch.zeros(n, rank + P, device=device)
        row[t, t % rank] = 1.0
        row[:, rank:] = z
        c.rows[table[b].to(device).long()[t // page], t % page] = row.to(c.rows.dtype)
        out.append(z)
    return c, out


def heads(dtype, lens, Hkv, D, page, seed, device, table):
    """A cache of key-value heads of such rows; and the codes [L, D] of each sequence and KV head."""
    B, cols = table.shape
    c = kvd.PagedKVCache(dtype, B, B * cols, Hkv, page, cols, head_dim=D, device=device)
    c.page_table.copy_(table)
    c.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
    c.len = max(lens)
    for x in ("k", "v"):
        if dtype == kvd.INT8:
            c.t[x].fill_(127)
            c.t[x + "_scale"].fill_(math.nan)
        else:
            c.t[x].fill_(math.nan)
    out = []
    for b, n in enumerate(lens):
        t = torch.arange(n, device=device)
        ids, at = table[b].to(device).long()[t // page], t % page
        out.append([])
        for g in range(Hkv):
            z = codes(n, D, seed + b * Hkv + g, device)
            v = torch.zeros(n, D, device=device)
            v[t, t % D] = 1.0
            c.k[ids, g, at] = z.to(c.k.dtype)
            c.v[ids, g, at] = v.to(c.v.dtype)
            if dtype == kvd.INT8:
                c.k_scale[ids, g, at] = 1.0
                c.v_scale[ids, g, at] = 1.0
            out[b].append(z)
    return c, out


def queries(pick, W, first, x, device):
    """Rows [T, H, W] that pick their channel (counted from `first`) of a key."""
    T, H = pick.shape
    q = torch.zeros(T, H, W, device=device)
    some = pick >= 0
    i, h = torch.nonzero(some, as_tuple=True)
    q[i.to(device), h.to(device), pick[some].to(device) + first] = 1.0
    return q.to(x)
