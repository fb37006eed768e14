"""The operators that keep a long context's cache small, as they are measured.

Four kinds of case:
  append  latent_append: norm of a token's latent vector, rotation of its shared key part, into pages; the
          queries' rotated part with it
  attn    latent_attn:   attention over the latent pages, in which a row is the key and its first channels the value
  mass    an attention call with its softmax statistics, then paged_mass: how much weight each cached token got,
          over a latent cache or one of key-value heads
  evict   paged_evict:   the tokens with most accumulated weight, the first and the last ones, moved to other pages

`run` computes the plain form (elementary torch operations, 32 bits, angles in 64) or, with `own`
set, makes the framework's calls.  `exact` computes the definition in 64 bits, sequence by sequence.
"""
import math

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
DEV = "cuda"


def _latent(name, kind, B, new, ctx, H, R, P, page, x, ragged=0, window=0, scaling="none", layout="half", norm=True,
            decay=1.0):
    return dict(name=name, kind=kind, cache="latent", B=B, new=new, ctx=ctx, H=H, R=R, P=P, page=page, x=x,
                ragged=ragged, window=window, scaling=scaling, layout=layout, norm=norm, decay=decay)


def _heads(name, B, new, ctx, H, Hkv, D, page, x, cache, ragged=0, window=0, decay=1.0):
    return dict(name=name, kind="mass", cache=cache, B=B, new=new, ctx=ctx, H=H, Hkv=Hkv, D=D, page=page, x=x,
                ragged=ragged, window=window, decay=decay)


def _evict(name, B, ctx, keep, sink, recent, Hkv, D, page, cache, ragged=0):
    return dict(name=name, kind="evict", cache=cache, B=B, ctx=ctx, keep=keep, sink=sink, recent=recent, Hkv=Hkv, D=D,
                page=page, ragged=ragged)


def listed():
    return [
        # a decode batch's new tokens of a layer with many heads: latency
        _latent("latent_append_64x1_bf16", "append", 64, 1, 2048, 128, 512, 64, 64, "bf16"),
        # two prompts' chunks, a stretched context: bytes
        _latent("latent_append_2x4095_f16", "append", 2, 4095, 0, 32, 512, 64, 64, "f16", scaling="yarn"),
        # the smallest attention: one token over a short context, 16 heads
        _latent("latent_decode_512_bf16", "attn", 1, 1, 511, 16, 512, 64, 64, "bf16"),
        # a decode batch with many heads: as many products as bytes
        _latent("latent_decode_32x8k_bf16", "attn", 32, 1, 8191, 128, 512, 64, 64, "bf16"),
        # few sequences over very long contexts: bound by the cache's bytes
        _latent("latent_decode_4x100k_f16", "attn", 4, 1, 99999, 32, 512, 64, 64, "f16"),
        # a prefill chunk behind a prompt: bound by the tensor cores
        _latent("latent_chunk_1000_over_8k_bf16", "attn", 1, 1000, 8000, 32, 512, 64, 64, "bf16"),
        # chunks, single tokens and all between in one batch, small pages, narrow rows, a sliding window
        _latent("latent_mixed_24_f16_window", "attn", 24, 256, 4000, 24, 256, 32, 16, "f16", ragged=1, window=1500),
        # a decode step that keeps count of each token's weight, over heads of keys and values
        _heads("mass_8x64k_f16", 8, 1, 65535, 32, 8, 128, 64, "f16", "f16"),
        # a prompt's chunk that does, over the 8-bit cache, older weights fading
        _heads("mass_chunk_1024_over_8k_int8", 1, 1024, 8000, 32, 8, 128, 64, "f16", "int8", decay=0.9),
        # a decode step that does, over latent rows
        _latent("mass_latent_16x16k_bf16", "mass", 16, 1, 16383, 64, 512, 64, 64, "bf16"),
        # a small cache cut to a quarter: latency
        _evict("evict_1x4k_to_1k_bf16", 1, 4096, 1024, 4, 256, 8, 128, 64, "bf16"),
        # a batch of long 8-bit caches cut to a quarter: bytes
        _evict("evict_8x64k_to_16k_int8", 8, 65536, 16384, 4, 1024, 8, 128, 64, "int8", ragged=1),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    kind = rng.choice(["append", "attn", "attn", "attn", "mass", "mass", "evict"])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    if kind == "evict":
        B = _log(rng, 1, 32)
        ctx = _log(rng, 64, min(100000, 400000 // B))
        keep = _log(rng, 32, ctx + 100)
        sink = rng.choice([0, 4, 4, keep // 4])
        c = _evict("", B, ctx, keep, sink, rng.choice([0, keep // 8, keep - sink]), rng.choice([1, 2, 4, 8]),
                   rng.choice([64, 128]), page, rng.choice(["f16", "bf16", "int8", "latent"]), int(rng.random() < 0.6))
        if c["cache"] == "latent":
            c.update(Hkv=1, D=rng.choice([512 + 64, 256 + 32, 128 + 64]))
        del c["name"]
        return c
    x = rng.choice(["f16", "bf16"])
    ragged, decay = int(rng.random() < 0.6), rng.choice([1.0, 0.95])
    window = 0 if kind == "append" or rng.random() < 0.7 else _log(rng, 1, 8000)
    B = _log(rng, 1, 32)
    new = _log(rng, 1, max(1, 2000 // B)) if rng.random() < 0.6 else 1
    if kind == "mass" and rng.random() < 0.6:
        Hkv = rng.choice([1, 2, 4, 8])
        ctx = _log(rng, 16, min(60000, 400000 // B, 8000000 // (B * new)))
        c = _heads("", B, new, ctx, Hkv * rng.choice([1, 2, 4, 7, 8]), Hkv, rng.choice([64, 128]), page, x,
                   rng.choice([x, x, "int8"]), ragged, window, decay)
    else:
        H = rng.choice([8, 16, 20, 32, 64, 96, 128])
        ctx = _log(rng, 16, min(100000, 250000 // B, 200000000 // (B * new * H)))
        c = _latent("", kind, B, new, ctx, H, rng.choice([128, 256, 512, 512]), rng.choice([32, 64, 64]), page, x,
                    ragged, window, rng.choice(["none", "linear", "yarn", "bands"]),
                    rng.choice(["half", "interleaved"]), rng.random() < 0.8, decay)
    del c["name"]
    return c


# ------------------------------------------------------------------ sizes ---

def _lengths(case):
    """(new tokens of each sequence, tokens cached with them), the same for every seed."""
    B, new, ctx = case["B"], case.get("new", 0), case["ctx"]
    if not case["ragged"]:
        return [new] * B, [ctx + new] * B
    u = [((b * 2654435761 + 12345) % 4294967296) / 4294967296 for b in range(2 * B)]
    # a third decode one token, the others have chunks of every length up to `new`; one sequence has no new token
    n = [0 if not new else 1 if b % 3 == 0 else max(1, int(new ** u[b])) for b in range(B)]
    n[0] = new
    if B > 2:
        n[2] = 0
    return n, [n[b] + int(ctx * (1.0 if b == 0 else u[B + b])) for b in range(B)]


def _kv_heads(case):
    return 1 if case["cache"] == "latent" else case["Hkv"]


def _width(case):
    """Channels of a cached key."""
    return case["D"] if "D" in case else case["R"] + case["P"]


def _scale(case):
    return (128 + case["P"]) ** -0.5 if "P" in case else case["D"] ** -0.5


def _freqs(case):
    """Angle per position of each channel pair, radians, in 64 bits; and the factor on the rotated channels."""
    r, base, s = case["P"], 10000.0, case["scaling"]
    factor, orig = 8.0, 8192.0
    i = torch.arange(r // 2, dtype=torch.float64, device=DEV)
    f = base ** (-2.0 * i / r)
    if s == "linear":
        return f / factor, 1.0
    if s == "bands":  # long waves slowed by the factor, short ones kept, a ramp between
        turns = orig * f / (2 * math.pi)
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        return f * (keep + (1.0 - keep) / factor), 1.0
    if s == "yarn":
        def at(turns):
            return r * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), r - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        return f * (1.0 - ramp + ramp / factor), 0.1 * math.log(factor) + 1.0
    return f, 1.0


# ------------------------------------------------------------------ inputs ---

def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _pool(g, case, shape, s):
    """Pages with data in every row."""
    if case["cache"] == "latent":
        x = TYPES[case.get("x", "bf16")]
        s["rows"] = torch.empty(shape[:1] + shape[2:], dtype=x, device=DEV).normal_(generator=g)
        return
    for a in "kv":
        if case["cache"] == "int8":
            s[a + "_pages"] = torch.randint(-127, 128, shape, generator=g, device=DEV, dtype=torch.int8)
            s[a + "_scale"] = torch.rand(shape[:3], generator=g, device=DEV) * 0.01 + 0.01
        else:
            s[a + "_pages"] = torch.empty(shape, dtype=TYPES[case["cache"]], device=DEV).normal_(generator=g)


def _inputs(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": case}
    n, lens = _lengths(case)
    B, page, Hkv, W = case["B"], case["page"], _kv_heads(case), _width(case)
    T, cols = sum(n), max((m + page - 1) // page for m in lens) + 1
    s["T"], s["max_new"], s["max_len"] = T, max(n), max(lens)
    s["lens"] = torch.tensor(lens, device=DEV).int()
    if case["kind"] == "evict":
        to = (case["keep"] + page - 1) // page
        ids = torch.randperm(B * (cols + to), generator=g, device=DEV).int()
        s["table"], s["to"] = ids[:B * cols].view(B, cols), ids[B * cols:].view(B, to)
        _pool(g, case, (B * (cols + to), Hkv, page, W), s)
        # a few tokens hold most of the weight, many have next to none, some (behind a window) none at all
        mass = torch.randn(B, Hkv, cols * page, generator=g, device=DEV).mul_(2.0).exp_()
        s["mass"] = mass.masked_fill_(torch.rand(mass.shape, generator=g, device=DEV) < 0.1, 0.0)
        return s
    n = torch.tensor(n, device=DEV)
    s["starts"] = torch.cat([n.new_zeros(1), n.cumsum(0)]).int()
    seq = torch.repeat_interleave(torch.arange(B, device=DEV), n, output_size=T)
    s["seq"] = seq
    s["row"] = torch.arange(T, device=DEV) - s["starts"].long()[seq]  # place among the sequence's new tokens
    s["pos"] = (s["lens"].long() - n)[seq] + s["row"]
    pages = B * cols
    s["table"] = torch.randperm(pages, generator=g, device=DEV).view(B, cols).int()
    _pool(g, case, (pages, Hkv, page, W), s)
    x = TYPES[case["x"]]
    if case["kind"] == "append":
        R, P, H = case["R"], case["P"], case["H"]
        down = _normal(g, (T, R + P), x)  # one projection's output: the latent and the shared key part
        s["c"], s["k_pe"] = down[:, :R], down[:, R:]
        s["q_pe"] = _normal(g, (T, H, 128 + P), x)[:, :, 128:]  # beside the queries' other channels
        if case["norm"]:
            s["cw"] = torch.rand(R, generator=g, device=DEV) + 0.5
    else:
        s["q"] = _normal(g, (T, case["H"], W), x)
    if case["kind"] == "mass":  # what earlier steps left, of the size of one step's
        s["mass"] = torch.rand(B, Hkv, cols * page, generator=g, device=DEV) * (case["H"] / Hkv / max(case["ctx"], 1))
    return s


def _value_width(case):
    return case["R"] if case["cache"] == "latent" else case["D"]


def prepare(case, seed):
    s = _inputs(case, seed)
    kind, B, Hkv = case["kind"], case["B"], _kv_heads(case)
    if kind == "append":
        s["q_out"] = torch.zeros(s["T"], case["H"], case["R"] + case["P"], dtype=s["c"].dtype, device=DEV)
        s["freqs"], s["mscale"] = _freqs(case)
    elif kind == "evict":
        s["kept"] = torch.full((B, Hkv, case["keep"]), -1, dtype=torch.int32, device=DEV)
        s["new_lens"] = torch.empty(B, dtype=torch.int32, device=DEV)
        s["new_mass"] = torch.zeros(B, Hkv, case["keep"], device=DEV)
    else:
        s["out"] = torch.empty(s["T"], case["H"], _value_width(case), dtype=s["q"].dtype, device=DEV)
    if kind == "mass":
        s["lse"] = torch.empty(s["T"], case["H"], device=DEV)
        s["new_mass"] = torch.zeros_like(s["mass"])
    if own:
        import long_context_decode_kv_gb300 as kvd
        if kind == "append":
            s["rope"] = kvd.rope_table(case["P"], 10000.0, interleaved=case["layout"] == "interleaved",
                                       scaling=case["scaling"], factor=8.0, orig_len=8192, device=DEV)
        t = {"page_table": s["table"], "seq_lens": s["lens"]}
        cols = s["table"].shape[1]
        if case["cache"] == "latent":
            t["rows"] = s["rows"]
            dtype = kvd.F16 if s["rows"].dtype == torch.float16 else kvd.BF16
            P = case.get("P", 32 if _width(case) == 288 else 64)
            s["cache"] = kvd.LatentCache(dtype, B, s["rows"].shape[0], case["page"], cols, rank=_width(case) - P,
                                         rope_dim=P, device=DEV, tensors=t)
        else:
            dtype = {"f16": kvd.F16, "bf16": kvd.BF16, "int8": kvd.INT8}[case["cache"]]
            t.update(k=s["k_pages"], v=s["v_pages"])
            if dtype == kvd.INT8:
                t.update(k_scale=s["k_scale"], v_scale=s["v_scale"])
            s["cache"] = kvd.PagedKVCache(dtype, B, s["k_pages"].shape[0], Hkv, case["page"], cols,
                                          head_dim=case["D"], device=DEV, tensors=t)
        s["cache"].len = s["max_len"]
        if kind in ("attn", "mass"):
            make = kvd.make_latent_workspace if case["cache"] == "latent" else kvd.make_paged_workspace
            s["ws"] = make(s["cache"], case["H"], s["T"], s["max_new"])
    return s


# -------------------------------------------------------------- plain form ---

def _turned(x, pos, freqs, mscale, layout):
    """x [T, heads, P] turned by its token's position, in f32."""
    x = x.float()
    a = pos.double()[:, None] * freqs
    c, s = (a.cos() * mscale).float()[:, None], (a.sin() * mscale).float()[:, None]
    if layout == "half":
        h = x.shape[-1] // 2
        u, v = x[..., :h], x[..., h:]
        return torch.cat([u * c - v * s, v * c + u * s], -1)
    u, v = x[..., 0::2], x[..., 1::2]
    return torch.stack([u * c - v * s, v * c + u * s], -1).flatten(-2)


def _append(s):
    case = s["case"]
    R, page = case["R"], case["page"]
    c = s["c"].float()
    if case["norm"]:
        c = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS) * s["cw"]
    turn = (s["pos"], s["freqs"], s["mscale"], case["layout"])
    row = torch.cat([c, _turned(s["k_pe"][:, None], *turn)[:, 0]], -1)
    s["rows"][s["table"].long()[s["seq"], s["pos"] // page], s["pos"] % page] = row.to(s["rows"].dtype)
    s["q_out"][..., R:] = _turned(s["q_pe"], *turn).to(s["q_out"].dtype)


def _gathered(s, name):
    """A cache side as [B, heads, tokens, channels] in f32."""
    table = s["table"].long()
    if name == "rows":
        return s["rows"][table].float().flatten(1, 2)[:, None]
    x = s[name + "_pages"][table].float()
    if s["case"]["cache"] == "int8":
        x = x * s[name + "_scale"][table][..., None]
    B, cols, Hkv, page, D = x.shape
    return x.transpose(1, 2).reshape(B, Hkv, cols * page, D)


def _attend(s):
    """(output, statistics, weight of each token) in f32."""
    case = s["case"]
    B, H, Hkv, n, W = case["B"], case["H"], _kv_heads(case), s["max_new"], _width(case)
    G = H // Hkv
    if case["cache"] == "latent":
        k = _gathered(s, "rows")
        v = k[..., :case["R"]]
    else:
        k, v = _gathered(s, "k"), _gathered(s, "v")
    L = k.shape[2]
    rows = torch.zeros(B, n, H, W, device=DEV)
    rows[s["seq"], s["row"]] = s["q"].float()
    pos = torch.full((B, n), -1, device=DEV)
    pos[s["seq"], s["row"]] = s["pos"]
    rows = rows.view(B, n, Hkv, G, W).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, W)
    t = torch.arange(L, device=DEV)
    seen = t <= pos[..., None]
    if case["window"]:
        seen &= t > pos[..., None] - case["window"]
    z = (rows @ k.transpose(2, 3)).view(B, Hkv, n, G, L) * _scale(case)
    z.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = z.amax(-1, keepdim=True).clamp_min(-1e30)
    z -= top
    z.exp_()
    total = z.sum(-1, keepdim=True)
    o = (z.view(B, Hkv, n * G, L) @ v).view(B, Hkv, n, G, v.shape[-1]) / total.clamp_min(1e-30)
    o = o.permute(0, 2, 1, 3, 4).reshape(B, n, H, v.shape[-1])[s["seq"], s["row"]]
    if case["kind"] == "attn":
        return o, None, None
    lse = torch.where(total > 0, top + total.log(), -math.inf)[..., 0]
    lse = lse.permute(0, 2, 1, 3).reshape(B, n, H)[s["seq"], s["row"]]
    z /= total.clamp_min(1e-30)
    return o, lse, z.sum((2, 3))


def _add_mass(s, weight):
    t = torch.arange(weight.shape[-1], device=DEV)
    n = (s["starts"][1:] - s["starts"][:-1])[:, None, None]
    lens = s["lens"][:, None, None]
    old = torch.where(t < lens - n, s["mass"] * s["case"]["decay"], 0.0)
    s["new_mass"].copy_(torch.where(t < lens, old + weight, s["new_mass"]))


def _drop(s):
    case = s["case"]
    mass, lens, keep, page = s["mass"], s["lens"].long(), case["keep"], case["page"]
    t = torch.arange(mass.shape[-1], device=DEV)
    l = lens[:, None, None]
    first = (t < case["sink"]) | (t >= l - case["recent"])
    rank = torch.where(first, math.inf, mass).masked_fill(t >= l, -math.inf)
    order = rank.sort(dim=-1, descending=True, stable=True).indices[..., :keep]
    n = lens.clamp_max(keep)
    some = (torch.arange(order.shape[-1], device=DEV) < n[:, None, None]).expand(order.shape)
    order = order.masked_fill(~some, mass.shape[-1]).sort(-1).values
    b, g, r = some.nonzero(as_tuple=True)
    old = order[b, g, r]
    s["kept"][b, g, r] = old.int()
    s["new_mass"][b, g, r] = mass[b, g, old]
    s["new_lens"].copy_(n)
    src, dst = s["table"].long()[b, old // page], s["to"].long()[b, r // page]
    if case["cache"] == "latent":
        s["rows"][dst, r % page] = s["rows"][src, old % page]
        return
    for name in ("k_pages", "v_pages") + (("k_scale", "v_scale") if case["cache"] == "int8" else ()):
        s[name][dst, g, r % page] = s[name][src, g, old % page]


def _evict_outputs(s):
    pools = [s[a] for a in ("rows", "k_pages", "v_pages", "k_scale", "v_scale") if a in s]
    return [s["kept"], s["new_lens"], s["new_mass"]] + pools


def run(state):
    s, case = state, state["case"]
    kind = case["kind"]
    if own:
        import long_context_decode_kv_gb300 as kvd
        if kind == "append":
            kvd.latent_append(s["cache"], s["c"], s["k_pe"], s["starts"], rope=s["rope"], c_weight=s.get("cw"),
                              eps=EPS, q_pe=s["q_pe"], q_out=s["q_out"])
            return s["q_out"], s["rows"]
        if kind == "evict":
            kvd.paged_evict(s["cache"], s["mass"], case["keep"], s["to"], s["kept"], s["new_lens"],
                            mass_out=s["new_mass"], sink=case["sink"], recent=case["recent"])
            return _evict_outputs(s)
        attn = kvd.latent_attn if case["cache"] == "latent" else kvd.paged_attn
        attn(s["cache"], s["q"], s["starts"], s["max_new"], _scale(case), s["out"], s["ws"], window=case["window"],
             lse=s.get("lse"))
        if kind == "attn":
            return s["out"]
        kvd.paged_mass(s["cache"], s["q"], s["lse"], s["starts"], s["max_new"], _scale(case), s["mass"],
                       out=s["new_mass"], decay=case["decay"], window=case["window"])
        return s["out"], s["lse"], s["new_mass"]
    if kind == "append":
        _append(s)
        return s["q_out"], s["rows"]
    if kind == "evict":
        _drop(s)
        return _evict_outputs(s)
    o, lse, weight = _attend(s)
    s["out"].copy_(o)
    if kind == "attn":
        return s["out"]
    s["lse"].copy_(lse)
    _add_mass(s, weight)
    return s["out"], s["lse"], s["new_mass"]


def work(case):
    size = {"f16": 2, "bf16": 2, "f32": 4, "int8": 1, "latent": 2}
    n, lens = _lengths(case)
    T, Hkv, W = sum(n), _kv_heads(case), _width(case)
    row = W * size[case["cache"]] + (4 if case["cache"] == "int8" else 0)
    sides = 1 if case["cache"] == "latent" else 2
    if case["kind"] == "append":
        x = size[case["x"]]
        return {"bytes": T * W * (x + 2) + 2 * T * case["H"] * case["P"] * x,
                "flops": 3 * T * (case["H"] + 1) * case["P"] + 4 * T * case["R"] * int(case["norm"])}
    if case["kind"] == "evict":
        kept = sum(min(case["keep"], m) for m in lens)
        return {"bytes": Hkv * (4 * sum(lens) + kept * (2 * sides * row + 8)), "flops": 0}
    w = case["window"] or 1 << 40
    pairs = tokens = 0
    for m, total in zip(n, lens):  # keys seen: position p sees min(p + 1, w) of them
        first = total - m
        full = max(0, min(total, w) - first)  # rows whose window is not full
        pairs += full * first + full * (full + 1) // 2 + (m - full) * (w if m > full else 0)
        tokens += min(total, w + m - 1) if m else 0
    V = _value_width(case)
    b = T * case["H"] * (W + V) * size[case["x"]] + sides * tokens * Hkv * row
    if case["kind"] == "mass":
        b += 8 * Hkv * sum(lens) + 4 * T * case["H"]
    return {"bytes": b, "flops": 2.0 * pairs * case["H"] * (W + V)}


# ------------------------------------------------------------------- exact ---

def _exact_turn(x, pos, case):
    """The rotation as a product with exp(i angle), in 64 bits; x [T, heads, P]."""
    f, m = _freqs(case)
    angle = torch.outer(pos.double(), f)
    z = torch.polar(torch.full_like(angle, m), angle)[:, None, :]
    x = x.double()
    half = case["layout"] == "half"
    pairs = x.unflatten(-1, (2, -1)).transpose(-1, -2) if half else x.unflatten(-1, (-1, 2))
    y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
    return (y.transpose(-1, -2) if half else y).flatten(-2)


def _exact_evict(s, case):
    B, Hkv, page, keep = case["B"], case["Hkv"], case["page"], case["keep"]
    kept = torch.full((B, Hkv, keep), -1, dtype=torch.int32, device=DEV)
    new_mass = torch.zeros(B, Hkv, keep, dtype=torch.float64, device=DEV)
    lens = s["lens"].tolist()
    names = [a for a in ("rows", "k_pages", "v_pages", "k_scale", "v_scale") if a in s]
    pools = {a: s[a].clone() for a in names}
    for b, total in enumerate(lens):
        n = min(total, keep)
        rows = torch.arange(n, device=DEV)
        to = s["to"][b].long()[rows // page] * page + rows % page
        for h in range(Hkv):
            if total <= keep:
                ids = rows
            else:
                lo, hi = case["sink"], total - case["recent"]
                m = s["mass"][b, h, lo:hi]
                by = torch.argsort(-m, stable=True)[:keep - case["sink"] - case["recent"]] + lo
                ends = [torch.arange(lo, device=DEV), torch.arange(hi, total, device=DEV)]
                ids = torch.cat([ends[0], by.sort().values, ends[1]])
            kept[b, h, :n] = ids.int()
            new_mass[b, h, :n] = s["mass"][b, h, ids].double()
            at = s["table"][b].long()[ids // page] * page + ids % page
            for a in names:
                if a == "rows":
                    pools[a].flatten(0, 1)[to] = s[a].flatten(0, 1)[at]
                else:
                    pools[a][to // page, h, to % page] = s[a][at // page, h, at % page]
    out = [pools[a] if pools[a].dtype == torch.int8 else pools[a].double() for a in names]
    return [kept, torch.tensor([min(m, keep) for m in lens], dtype=torch.int32, device=DEV), new_mass] + out


def exact(case, seed):
    if work(case)["flops"] > 3e12:  # the 64-bit products alone would take too long
        return None
    s = _inputs(case, seed)
    kind = case["kind"]
    if kind == "evict":
        return _exact_evict(s, case)
    n, lens = _lengths(case)
    page, H, Hkv, W = case["page"], case["H"], _kv_heads(case), _width(case)
    if kind == "append":
        R = case["R"]
        c = s["c"].double()
        if case["norm"]:
            c = c / torch.sqrt((c ** 2).sum(-1, keepdim=True) / R + EPS) * s["cw"].double()
        rows = s["rows"].double()
        at = s["table"].long()[s["seq"], s["pos"] // page], s["pos"] % page
        rows[at] = torch.cat([c, _exact_turn(s["k_pe"][:, None], s["pos"], case)[:, 0]], -1)
        q = torch.zeros(s["T"], H, W, dtype=torch.float64, device=DEV)
        q[..., R:] = _exact_turn(s["q_pe"], s["pos"], case)
        return q, rows
    G, V = H // Hkv, _value_width(case)
    out = torch.zeros(s["T"], H, V, dtype=torch.float64, device=DEV)
    lse = torch.full((s["T"], H), -math.inf, dtype=torch.float64, device=DEV)
    mass = torch.zeros(s["mass"].shape, dtype=torch.float64, device=DEV) if kind == "mass" else None
    first = 0
    for b, (m, total) in enumerate(zip(n, lens)):
        if mass is not None:
            mass[b, :, :total - m] = s["mass"][b, :, :total - m].double() * case["decay"]
        if m:
            ids = s["table"][b, :(total + page - 1) // page].long()
            p = torch.arange(total - m, total, device=DEV)
            old = torch.arange(total, device=DEV)
            seen = old[None, :] <= p[:, None]
            if case["window"]:
                seen = seen & (p[:, None] - old[None, :] < case["window"])
            for g in range(Hkv):
                if case["cache"] == "latent":
                    k = s["rows"][ids].double().flatten(0, 1)[:total]
                    v = k[:, :V]
                else:
                    side = []
                    for a in "kv":
                        x = s[a + "_pages"][ids, g].double()
                        if case["cache"] == "int8":
                            x = x * s[a + "_scale"][ids, g].double()[..., None]
                        side.append(x.reshape(-1, W)[:total])
                    k, v = side
                for h in range(g * G, g * G + G):
                    z = torch.where(seen, s["q"][first:first + m, h].double() @ k.T * _scale(case), -math.inf)
                    p_h = torch.softmax(z, -1)
                    out[first:first + m, h] = p_h @ v
                    if mass is not None:
                        lse[first:first + m, h] = torch.logsumexp(z, -1)
                        mass[b, g, :total] += p_h.sum(0)
        first += m
    return out if kind == "attn" else (out, lse, mass)
