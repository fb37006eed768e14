"""The operators around the paged cache, as they are measured.

Four kinds of case:
  rope    qk_norm_rope: per-head RMS norm (optional) and position rotation of queries and keys
  append  paged_append: keys (normed, rotated) and values into the pages, queries rotated in the same call
  attn    paged_attn:   attention of each sequence's new tokens over its pages
  step    paged_append, then paged_attn: one layer's share of a decode step or of a chunk

`run` computes the plain form (elementary torch operations, 32 bits, angles in 64) or, with `own`
set, makes the framework's calls.  `exact` computes the definition in 64 bits, sequence by sequence.
"""
import math

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
DEV = "cuda"


def _rope(name, T, H, Hkv, D, rot, layout, scaling, norm, x, q_out, k_out, far=0):
    return dict(name=name, kind="rope", T=T, H=H, Hkv=Hkv, D=D, rot=rot, layout=layout, scaling=scaling,
                norm=norm, x=x, q_out=q_out, k_out=k_out, far=far)


def _paged(name, kind, B, new, ctx, H, Hkv, D, page, x, cache, ragged=0, window=0, rot=0, layout="half",
           scaling="none", norm=False):
    return dict(name=name, kind=kind, B=B, new=new, ctx=ctx, H=H, Hkv=Hkv, D=D, page=page, x=x, cache=cache,
                ragged=ragged, window=window, rot=rot, layout=layout, scaling=scaling, norm=norm)


def listed():
    return [
        # one token of one sequence in front of a decode step (f32 queries, f16 keys, as that call takes them): latency
        _rope("rope_token_f16", 1, 32, 8, 128, 128, "half", "none", False, "f16", "f32", "f16", far=32768),
        # a long chunk of a model with per-head norms, at far positions of a stretched context
        _rope("norm_rope_8k_bf16", 8192, 32, 8, 128, 128, "half", "yarn", True, "bf16", "bf16", "bf16", far=1000000),
        # an odd number of tokens, a quarter of a small head rotated in interleaved pairs, 32-bit activations
        _rope("rope_part_f32_d64", 1021, 8, 8, 64, 16, "interleaved", "linear", False, "f32", "f32", "f32"),
        # a decode batch: one token for each of 64 sequences, small pages
        _paged("append_64x1_f16", "append", 64, 1, 2048, 32, 8, 128, 16, "f16", "f16", rot=128),
        # a prefill batch: two sequences' chunks into pages of one block
        _paged("append_2x4095_bf16", "append", 2, 4095, 0, 32, 8, 128, 64, "bf16", "bf16", rot=128,
               scaling="bands", norm=True),
        # the smallest attention: one token over a short context, one query head per KV head
        _paged("decode_512_f16", "attn", 1, 1, 511, 8, 8, 128, 64, "f16", "f16"),
        # a decode batch over a long 8-bit cache: bound by the cache's bytes
        _paged("decode_8x128k_int8", "attn", 8, 1, 131071, 32, 8, 128, 64, "f16", "int8"),
        # a prefill chunk in the middle of a long prompt: bound by the tensor cores
        _paged("chunk_2k_over_32k_f16", "attn", 1, 2048, 30720, 32, 8, 128, 64, "f16", "f16"),
        # chunks, single tokens and all between in one batch, small pages, a sliding window
        _paged("mixed_24_bf16_window", "attn", 24, 512, 6000, 32, 8, 128, 16, "bf16", "bf16", ragged=1, window=4096),
        # whole prompts of a model with small heads, not a round number of tokens
        _paged("prefill_2x4001_bf16_d64", "attn", 2, 4001, 0, 16, 4, 64, 32, "bf16", "bf16"),
        # a short chunk over a very long 8-bit cache
        _paged("chunk_250_over_128k_int8", "attn", 1, 250, 130000, 32, 8, 128, 64, "f16", "int8"),
        # one layer's decode step on the 8-bit cache: norm, rotation, quantisation, attention
        _paged("step_4x32k_int8", "step", 4, 1, 32000, 32, 8, 128, 64, "f16", "int8", rot=128, norm=True),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    kind = rng.choice(["rope", "append", "attn", "attn", "attn", "step"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([1, 2, 4, 7, 8])
    rot = rng.choice([D, D, D // 2, 16])
    layout = rng.choice(["half", "half", "interleaved"])
    scaling = rng.choice(["none", "linear", "ntk", "yarn", "bands"])
    norm = rng.random() < 0.5
    if kind == "rope":
        x = rng.choice(["f16", "bf16", "f32"])
        c = _rope("", _log(rng, 1, 8000), H, Hkv, D, rot, layout, scaling, norm, x, rng.choice([x, "f32"]), x,
                  far=rng.choice([0, 1000, 1000000]))
    else:
        x = rng.choice(["f16", "bf16"])
        cache = x if kind == "append" else rng.choice([x, x, "int8"])
        page = rng.choice([16, 32, 48, 64, 128, 256])
        B = _log(rng, 1, 32)
        new = _log(rng, 1, max(1, 4000 // B)) if rng.random() < 0.7 else 1
        if kind == "append":
            ctx = _log(rng, 1, 2000)
        else:  # at most a quarter of the largest cases' bytes and products
            ctx = _log(rng, 16, min(100000, 400000 // B, 40000000 // (B * new)))
        c = _paged("", kind, B, new, ctx, H, Hkv, D, page, x, cache, ragged=int(rng.random() < 0.6),
                   window=0 if kind == "append" or rng.random() < 0.7 else _log(rng, 1, 8000))
        if kind != "attn":
            c.update(rot=rot, layout=layout, scaling=scaling, norm=norm)
    del c["name"]
    return c


# ------------------------------------------------------------------ sizes ---

def _lengths(case, seed=0):
    """(new tokens of each sequence, tokens cached with them), the same for every seed."""
    B, new, ctx = case["B"], case["new"], case["ctx"]
    if not case["ragged"]:
        return [new] * B, [ctx + new] * B
    u = [((b * 2654435761 + 12345) % 4294967296) / 4294967296 for b in range(2 * B)]
    # a third decode one token, the others have chunks of every length up to `new`; one sequence has no new token
    n = [1 if b % 3 == 0 else max(1, int(new ** u[b])) for b in range(B)]
    n[0] = new
    if B > 2:
        n[2] = 0
    return n, [n[b] + int(ctx * (1.0 if b == 0 else u[B + b])) for b in range(B)]


def _freqs(case):
    """Angle per position of each channel pair, radians, in 64 bits; and the factor on the rotated channels."""
    r, base, s = case["rot"], 10000.0, case["scaling"]
    factor, orig = 8.0, 8192.0
    i = torch.arange(r // 2, dtype=torch.float64, device=DEV)
    if s == "ntk":
        base = base * factor ** (r / (r - 2.0))
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


def _inputs(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    H, Hkv, D = case["H"], case["Hkv"], case["D"]
    x = TYPES[case["x"]]
    s = {"case": case}
    if case["kind"] == "rope":
        T = case["T"]
        qkv = _normal(g, (T, H + 2 * Hkv, D), x)  # one projection's output: queries, keys and values side by side
        s["q"], s["k"] = qkv[:, :H], qkv[:, H:H + Hkv]
        s["pos"] = (torch.arange(T, device=DEV) + case["far"] + torch.randint(0, 64, (1,), generator=g, device=DEV)).int()
    else:
        n, lens = _lengths(case)
        B, page = case["B"], case["page"]
        T, cols = sum(n), max((m + page - 1) // page for m in lens) + 1
        qkv = _normal(g, (T, H + 2 * Hkv, D), x)
        s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        s["T"], s["max_new"], s["max_len"] = T, max(n), max(lens)
        n = torch.tensor(n, device=DEV)
        s["lens"] = torch.tensor(lens, device=DEV).int()
        s["starts"] = torch.cat([n.new_zeros(1), n.cumsum(0)]).int()
        seq = torch.repeat_interleave(torch.arange(B, device=DEV), n, output_size=T)
        s["seq"] = seq
        s["row"] = torch.arange(T, device=DEV) - s["starts"].long()[seq]  # place among the sequence's new tokens
        s["pos"] = (s["lens"].long() - n)[seq] + s["row"]
        pages = B * cols
        s["table"] = torch.randperm(pages, generator=g, device=DEV).view(B, cols).int()
        shape = (pages, Hkv, page, D)
        if case["cache"] == "int8":
            for a in "kv":
                s[a + "_pages"] = torch.randint(-127, 128, shape, generator=g, device=DEV, dtype=torch.int8)
                s[a + "_scale"] = torch.rand(shape[:3], generator=g, device=DEV) * 0.01 + 0.01
        else:
            for a in "kv":
                s[a + "_pages"] = torch.empty(shape, dtype=TYPES[case["cache"]], device=DEV).normal_(generator=g)
        if case["kind"] == "attn":  # the queries come rotated, in rows of their own
            s["q"] = s["q"].contiguous()
    if case.get("norm"):
        s["qw"] = torch.rand(D, generator=g, device=DEV) + 0.5
        s["kw"] = torch.rand(D, generator=g, device=DEV) + 0.5
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    kind, q, k = case["kind"], s["q"], s["k"]
    if kind == "rope":
        s["q_out"] = torch.empty(q.shape, dtype=TYPES[case["q_out"]], device=DEV)
        s["k_out"] = torch.empty(k.shape, dtype=TYPES[case["k_out"]], device=DEV)
    else:
        s["q_out"] = torch.empty(q.shape, dtype=q.dtype, device=DEV)
        s["out"] = torch.empty(q.shape, dtype=q.dtype, device=DEV)
    if case.get("rot"):
        s["freqs"], s["mscale"] = _freqs(case)
    if own:
        import long_context_decode_kv_gb300 as kvd
        if case.get("rot"):
            s["rope"] = kvd.rope_table(case["rot"], 10000.0, interleaved=case["layout"] == "interleaved",
                                       scaling=case["scaling"], factor=8.0, orig_len=8192, device=DEV)
        if kind != "rope":
            dtype = {"f16": kvd.F16, "bf16": kvd.BF16, "int8": kvd.INT8}[case["cache"]]
            t = {"k": s["k_pages"], "v": s["v_pages"], "page_table": s["table"], "seq_lens": s["lens"]}
            if dtype == kvd.INT8:
                t.update(k_scale=s["k_scale"], v_scale=s["v_scale"])
            s["cache"] = kvd.PagedKVCache(dtype, case["B"], s["table"].numel(), case["Hkv"], case["page"],
                                          s["table"].shape[1], head_dim=case["D"], device=DEV, tensors=t)
            s["cache"].len = s["max_len"]
            if kind != "append":
                s["ws"] = kvd.make_paged_workspace(s["cache"], case["H"], s["T"], s["max_new"])
    return s


# -------------------------------------------------------------- plain form ---

def _turned(x, w, pos, freqs, mscale, layout, rot):
    """Norm (where there is a weight) and rotation of x [T, heads, D], in f32."""
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    if not rot:
        return x
    a = pos.double()[:, None] * freqs
    c, s = (a.cos() * mscale).float()[:, None], (a.sin() * mscale).float()[:, None]
    if layout == "half":
        u, v = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([u * c - v * s, v * c + u * s], -1)
    else:
        u, v = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([u * c - v * s, v * c + u * s], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _turned_by(s, x, w):
    case = s["case"]
    return _turned(x, s.get(w), s["pos"], s.get("freqs"), s.get("mscale"), case["layout"], case["rot"])


def _store(s, name, x):
    """Rows x [T, Hkv, D] (f32) into their pages."""
    page = s["case"]["page"]
    at = s["table"].long()[s["seq"], s["pos"] // page], slice(None), s["pos"] % page
    if s["case"]["cache"] == "int8":
        scale = x.abs().amax(-1) / 127.0
        code = torch.where(scale[..., None] > 0, x / scale[..., None], 0.0).round().clamp(-127, 127)
        s[name + "_pages"][at] = code.to(torch.int8)
        s[name + "_scale"][at] = scale
    else:
        s[name + "_pages"][at] = x.to(s[name + "_pages"].dtype)


def _append(s):
    s["q_out"].copy_(_turned_by(s, s["q"], "qw"))
    _store(s, "k", _turned_by(s, s["k"], "kw"))
    _store(s, "v", s["v"].float())


def _gathered(s, name):
    """A cache side as [B, Hkv, tokens, D] in f32."""
    x = s[name + "_pages"][s["table"].long()].float()
    if s["case"]["cache"] == "int8":
        x = x * s[name + "_scale"][s["table"].long()][..., None]
    B, cols, Hkv, page, D = x.shape
    return x.transpose(1, 2).reshape(B, Hkv, cols * page, D)


def _attend(s, q):
    case = s["case"]
    B, H, Hkv, D, n = case["B"], case["H"], case["Hkv"], case["D"], s["max_new"]
    G = H // Hkv
    k, v = _gathered(s, "k"), _gathered(s, "v")
    L = k.shape[2]
    rows = torch.zeros(B, n, H, D, device=DEV)
    rows[s["seq"], s["row"]] = q.float()
    pos = torch.full((B, n), -1, device=DEV)
    pos[s["seq"], s["row"]] = s["pos"]
    rows = rows.view(B, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, D)
    t = torch.arange(L, device=DEV)
    seen = t <= pos[..., None]
    if case["window"]:
        seen &= t > pos[..., None] - case["window"]
    z = (rows @ k.transpose(2, 3)).view(B, Hkv, n, G, L) * D ** -0.5
    z.masked_fill_(~seen[:, None, :, None], -math.inf)
    z -= z.amax(-1, keepdim=True).clamp_min(-1e30)
    z.exp_()
    total = z.sum(-1)
    o = (z.view(B, Hkv, n * G, L) @ v).view(B, Hkv, n, G, D) / total.clamp_min(1e-30)[..., None]
    return o.permute(0, 2, 1, 3, 4).reshape(B, n, H, D)[s["seq"], s["row"]]


def run(state):
    s, case = state, state["case"]
    kind = case["kind"]
    if own:
        import long_context_decode_kv_gb300 as kvd
        if kind == "rope":
            kvd.qk_norm_rope(s["q"], s["k"], s["pos"], s["rope"], s["q_out"], s["k_out"],
                             q_weight=s.get("qw"), k_weight=s.get("kw"), eps=EPS)
            return s["q_out"], s["k_out"]
        if kind != "attn":
            kvd.paged_append(s["cache"], s["k"], s["v"], s["starts"], rope=s["rope"], q=s["q"], q_out=s["q_out"],
                             q_weight=s.get("qw"), k_weight=s.get("kw"), eps=EPS)
        if kind == "append":
            return s["q_out"], s["k_pages"], s["v_pages"]
        kvd.paged_attn(s["cache"], s["q"] if kind == "attn" else s["q_out"], s["starts"], s["max_new"],
                       case["D"] ** -0.5, s["out"], s["ws"], window=case["window"])
        return s["out"]
    if kind == "rope":
        return s["q_out"].copy_(_turned_by(s, s["q"], "qw")), s["k_out"].copy_(_turned_by(s, s["k"], "kw"))
    if kind != "attn":
        _append(s)
    if kind == "append":
        return s["q_out"], s["k_pages"], s["v_pages"]
    return s["out"].copy_(_attend(s, s["q"] if kind == "attn" else s["q_out"]))


def work(case):
    size = {"f16": 2, "bf16": 2, "f32": 4, "int8": 1}
    H, Hkv, D = case["H"], case["Hkv"], case["D"]
    if case["kind"] == "rope":
        T = case["T"]
        return {"bytes": T * D * (H * (size[case["x"]] + size[case["q_out"]]) +
                                  Hkv * (size[case["x"]] + size[case["k_out"]])) + 4 * T,
                "flops": 6 * T * (H + Hkv) * case["rot"] + 4 * T * (H + Hkv) * D * int(case["norm"])}
    n, lens = _lengths(case)
    T, row = sum(n), D * size[case["cache"]] + (4 if case["cache"] == "int8" else 0)
    b = f = 0.0
    if case["kind"] != "attn":
        b += T * D * size[case["x"]] * 2 * (H + Hkv) + 2 * T * Hkv * row
        f += 6 * T * (H + Hkv) * case["rot"]
    if case["kind"] != "append":
        w = case["window"] or 1 << 40
        pairs = tokens = 0
        for m, total in zip(n, lens):  # keys seen: position p sees min(p + 1, w) of them
            first = total - m
            full = max(0, min(total, w) - first)  # rows whose window is not full
            pairs += full * first + full * (full + 1) // 2 + (m - full) * (w if m > full else 0)
            tokens += min(total, w + m - 1) if m else 0
        b += 2 * T * H * D * size[case["x"]] + 2 * tokens * Hkv * row
        f += 4.0 * pairs * H * D
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------- exact ---

def _exact_turn(x, w, pos, case):
    """The rotation as a product with exp(i angle), in 64 bits."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
    r = case["rot"]
    if not r:
        return x
    f, m = _freqs(case)
    angle = torch.outer(pos.double(), f)
    z = torch.polar(torch.full_like(angle, m), angle)[:, None, :]
    part = x[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2) if case["layout"] == "half" else \
        x[..., :r].unflatten(-1, (r // 2, 2))
    y = torch.view_as_real(torch.view_as_complex(part.contiguous()) * z)
    y = y.transpose(-1, -2).flatten(-2) if case["layout"] == "half" else y.flatten(-2)
    return torch.cat([y, x[..., r:]], -1)


def exact(case, seed):
    if work(case)["flops"] > 3e12:  # the 64-bit products alone would take too long
        return None
    s = _inputs(case, seed)
    kind = case["kind"]
    if kind == "rope":
        return [_exact_turn(s[a], s.get(a + "w"), s["pos"], case) for a in "qk"]
    n, lens = _lengths(case)
    H, Hkv, page, D = case["H"], case["Hkv"], case["page"], case["D"]
    G = H // Hkv
    q = s["q"].double()
    fresh = {}
    if kind != "attn":
        q = _exact_turn(s["q"], s.get("qw"), s["pos"], case)
        fresh = {"k": _exact_turn(s["k"], s.get("kw"), s["pos"], case), "v": s["v"].double()}
        at = s["table"].long()[s["seq"], s["pos"] // page], slice(None), s["pos"] % page
        if kind == "append":
            pages = []
            for a in "kv":
                whole = s[a + "_pages"].double()
                whole[at] = fresh[a]
                pages.append(whole)
            return q, pages[0], pages[1]
        q = q.to(TYPES[case["x"]]).double()  # a step hands its queries on in their own type
        for a in "kv":  # and its cache holds rows in the cache's type
            if case["cache"] == "int8":
                scale = (fresh[a].abs().amax(-1) / 127.0).float()
                fresh[a] = (fresh[a] / scale.double()[..., None]).round().clamp(-127, 127) * scale.double()[..., None]
            else:
                fresh[a] = fresh[a].to(TYPES[case["cache"]]).double()
    out = torch.zeros(s["T"], H, D, dtype=torch.float64, device=DEV)
    first = 0
    for b, (m, total) in enumerate(zip(n, lens)):
        if m:
            ids = s["table"][b, :(total + page - 1) // page].long()
            p = torch.arange(total - m, total, device=DEV)
            old = torch.arange(total, device=DEV)
            seen = old[None, :] <= p[:, None]
            if case["window"]:
                seen = seen & (p[:, None] - old[None, :] < case["window"])
            for g in range(Hkv):
                side = {}
                for a in "kv":
                    x = s[a + "_pages"][ids, g].double()
                    if case["cache"] == "int8":
                        x = x * s[a + "_scale"][ids, g].double()[..., None]
                    x = x.reshape(-1, D)[:total].clone()
                    if fresh:
                        x[total - m:] = fresh[a][first:first + m, g]
                    side[a] = x
                for h in range(g * G, g * G + G):
                    z = torch.where(seen, q[first:first + m, h] @ side["k"].T / math.sqrt(D), -math.inf)
                    out[first:first + m, h] = torch.softmax(z, -1) @ side["v"]
        first += m
    return out
