"""Cases of the nested KV cache's serving operators: rotary positions, the
cache's rows (rotate, pack, read back), attention of a batch over one shared
prefix and each sequence's own tokens, the attention weight each cached token
has received, and eviction by it.

``run`` computes a case in plain torch operations (``own`` false) or with the
calls a user makes of the library (``own`` true) on what ``prepare`` gives.
The cache is the library's: a row is one token and one KV head, 128 values as
two planes of unsigned nibbles and an fp16 scale; the draft is (hi - 8) s, the
target (16 (hi - 8) + (lo - 8)) s / 16.
"""
import math

import torch

own = False

DEV = "cuda"
D = 128  # head dimension of the cache
RSD = 1.0 / math.sqrt(D)


def listed():
    return [
        # one verify pass's queries: fp32 columns of the fused q|k|v output, Llama-3-8B heads
        {"name": "rope_verify", "op": "rope", "tokens": 4, "heads": 32, "dim": 128, "rot": 128,
         "layout": "half", "src": "f32", "dst": "f16", "row": 6144, "base": 500000.0,
         "scaling": "none", "far": 8192, "inverse": False},
        # a long prompt's queries, adjacent pairs, half of the head, positions scaled for 8 x the context
        {"name": "rope_prompt", "op": "rope", "tokens": 8192, "heads": 32, "dim": 128, "rot": 64,
         "layout": "pairs", "src": "f16", "dst": "f16", "row": 4096, "base": 10000.0,
         "scaling": "yarn", "far": 65536, "inverse": False},
        # a verify step's keys and values of 32 sequences into their caches
        {"name": "append_verify", "op": "append", "batch": 32, "new": 4, "hkv": 8, "cap": 2048,
         "rot": 128, "layout": "half", "src": "f32", "base": 500000.0, "scaling": "bands",
         "far": 131072, "mode": 1},
        # a shared prompt's keys and values, once
        {"name": "append_prompt", "op": "append", "batch": 1, "new": 16384, "hkv": 8, "cap": 16384,
         "rot": 128, "layout": "half", "src": "f16", "base": 500000.0, "scaling": "none",
         "far": 16384, "mode": 1},
        # two streams drafting over one prompt: the smallest call, latency
        {"name": "attend_draft_few", "op": "attend", "batch": 2, "queries": 1, "heads": 32, "hkv": 8,
         "prefix": 2048, "cap": 128, "mode": 0},
        # ragged batch with eight query heads to a KV head, odd lengths, empty sequences
        {"name": "attend_draft_ragged", "op": "attend", "batch": 37, "queries": 1, "heads": 16,
         "hkv": 2, "prefix": 5003, "cap": 3001, "mode": 0},
        # a verify pass (three draft tokens and one more) of 16 streams
        {"name": "attend_verify", "op": "attend", "batch": 16, "queries": 4, "heads": 32, "hkv": 8,
         "prefix": 8192, "cap": 1024, "mode": 1},
        # the same of 128 streams over a long system prompt: the largest
        {"name": "attend_verify_wide", "op": "attend", "batch": 128, "queries": 4, "heads": 32,
         "hkv": 8, "prefix": 16384, "cap": 512, "mode": 1},
        # what a verify pass looked at in each stream's own tokens
        {"name": "weights_own", "op": "weights", "shared": False, "batch": 16, "queries": 4,
         "heads": 32, "hkv": 8, "tokens": 4096, "mode": 1},
        # what all streams looked at in the shared prompt
        {"name": "weights_shared", "op": "weights", "shared": True, "batch": 64, "queries": 4,
         "heads": 32, "hkv": 8, "tokens": 16384, "mode": 1},
        # a small cache cut to half
        {"name": "evict_half", "op": "evict", "batch": 4, "hkv": 8, "tokens": 1025, "keep": 512,
         "sinks": 4, "recent": 128},
        # a batch of long contexts cut to a quarter
        {"name": "evict_long", "op": "evict", "batch": 16, "hkv": 8, "tokens": 32768, "keep": 8192,
         "sinks": 4, "recent": 1024},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "weights", "evict"])
    scaling = rng.choice(["none", "linear", "ntk", "bands", "yarn"])
    if op == "rope":
        dim = rng.choice([64, 80, 96, 128, 256])
        heads = rng.randint(1, 40)
        tokens = min(_log(rng, 1, 8192), 8192 * 32 * 128 // (heads * dim))
        return {"op": op, "tokens": tokens, "heads": heads, "dim": dim,
                "rot": dim // rng.choice([1, 2, 4]), "layout": rng.choice(["half", "pairs"]),
                "src": rng.choice(["f16", "f32"]), "dst": rng.choice(["f16", "f32"]),
                "row": heads * dim + rng.choice([0, 1, 8, 2 * dim]),
                "base": rng.choice([10000.0, 500000.0]), "scaling": scaling,
                "far": _log(rng, 64, 1 << 20), "inverse": rng.random() < 0.3}
    hkv = rng.choice([1, 2, 4, 8])
    if op == "append":
        batch = _log(rng, 1, 64)
        new = min(_log(rng, 1, 16384), 16384 // batch)
        return {"op": op, "batch": batch, "new": new, "hkv": hkv, "cap": new + rng.randint(0, 1000),
                "rot": rng.choice([128, 64, 32]), "layout": rng.choice(["half", "pairs"]),
                "src": rng.choice(["f16", "f32"]), "base": rng.choice([10000.0, 500000.0]),
                "scaling": scaling, "far": _log(rng, 64, 1 << 20), "mode": rng.randint(0, 1)}
    if op == "evict":
        batch = _log(rng, 1, 16)
        tokens = _log(rng, 16, 32768)
        keep = rng.randint(max(1, tokens // 8), max(2, tokens // 2))
        sinks = rng.randint(0, min(8, keep))
        return {"op": op, "batch": batch, "hkv": hkv, "tokens": tokens, "keep": keep,
                "sinks": sinks, "recent": rng.randint(0, keep - sinks)}
    heads = hkv * rng.choice([1, 2, 4, 8])
    batch, queries, mode = _log(rng, 1, 128), rng.randint(1, 8), rng.randint(0, 1)
    if op == "weights":
        shared = rng.random() < 0.5
        tokens = _log(rng, 1, 16384 if shared else 4096)
        if not shared:
            batch = min(batch, 16)
        else:
            batch = max(1, min(batch, 64 * 4 * 32 // (queries * heads)))
        return {"op": op, "shared": shared, "batch": batch, "queries": queries, "heads": heads,
                "hkv": hkv, "tokens": tokens, "mode": mode}
    batch = max(1, min(batch, 128 * 4 * 32 // (queries * heads)))
    return {"op": op, "batch": batch, "queries": queries, "heads": heads, "hkv": hkv,
            "prefix": rng.choice([0, 1]) if rng.random() < 0.1 else _log(rng, 16, 16384),
            "cap": min(_log(rng, 1, 4096), 128 * 512 // batch), "mode": mode}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _ints(g, lo, hi, *shape):
    """int32 in lo .. hi."""
    return torch.randint(lo, hi + 1, shape, generator=g, device=DEV, dtype=torch.int32)


def _frequencies(rot, base, scaling):
    """(radians per position of the rot / 2 pairs as Python floats, magnitude)."""
    s, trained = 8.0, 8192
    if scaling == "ntk":
        base = base * s ** (rot / (rot - 2))
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        return [x / s for x in f], 1.0
    if scaling == "bands":  # by wavelength: short ones stay, long ones are divided by s
        out = []
        for x in f:
            t = (trained * x / (2 * math.pi) - 1.0) / (4.0 - 1.0)
            t = min(1.0, max(0.0, t))
            out.append(x * (t + (1.0 - t) / s))
        return out, 1.0
    if scaling == "yarn":  # by pair: a ramp from the pair with 32 turns to the one with 1
        def pair(turns):
            return rot * math.log(trained / (2 * math.pi * turns)) / (2 * math.log(base))
        low, high = max(0, math.floor(pair(32.0))), min(rot - 1, math.ceil(pair(1.0)))
        ramp = [min(1.0, max(0.0, (i - low) / max(high - low, 1e-3))) for i in range(rot // 2)]
        return [x * (1.0 - r + r / s) for x, r in zip(f, ramp)], 0.1 * math.log(s) + 1.0
    return f, 1.0


def _phases(freq):
    """Turns per position in units of 2^-64, as int64."""
    p = [round(x / (2 * math.pi) * 2.0 ** 64) % (1 << 64) for x in freq]
    return torch.tensor([x - (1 << 64) if x >> 63 else x for x in p], dtype=torch.int64, device=DEV)


def _rotation(case):
    freq, mag = _frequencies(case["rot"], case["base"], case["scaling"])
    return {"freq": torch.tensor(freq, dtype=torch.float64, device=DEV), "mag": mag,
            "phases": _phases(freq)}


def _pack(x):
    """fp16 rows [..., 128] as (hi, lo, scale)."""
    x = x.float()
    s = (x.abs().amax(-1) / 7.0).half()
    t = torch.where((s == 0)[..., None], torch.zeros_like(x), x / s.float()[..., None])
    q = torch.round(t)
    r = torch.round(16.0 * (t - q)).clamp(-8, 7)
    hi, lo = (q + 8).to(torch.uint8), (r + 8).to(torch.uint8)
    return (hi[..., 0::2] | (hi[..., 1::2] << 4), lo[..., 0::2] | (lo[..., 1::2] << 4), s)


def _keys(g, *shape):
    """Rows with a few strong channels, as keys have."""
    x = _normal(g, *shape, D) * 0.8
    x[..., 5] += 2.0
    x[..., 70] *= 3.0
    return x.half()


def _cache(g, *shape):
    """(k planes, v planes) of a cache of rows `shape`."""
    return _pack(_keys(g, *shape)), _pack(_normal(g, *shape, D).half())


def _lengths(g, batch, cap):
    """Ragged lengths: most anywhere in 0 .. cap, the first full, the last empty where there are several."""
    n = _ints(g, 0, cap, batch)
    n[0] = cap
    if batch > 2:
        n[-1] = 0
    return n


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    if op == "rope":
        st = _rotation(case)
        m, h, d, row = case["tokens"], case["heads"], case["dim"], case["row"]
        x = _normal(g, m * row) * 1.5
        x = x.half() if case["src"] == "f16" else x
        st["x"] = x.as_strided((m, h, d), (row, d, 1))
        st["pos"] = _ints(g, 0, case["far"] - 1, m)
    elif op == "append":
        st = _rotation(case)
        b, n, h, cap = case["batch"], case["new"], case["hkv"], case["cap"]
        kv = torch.cat([_keys(g, b, n, h).float(), _normal(g, b, n, h, D)], 2)
        kv = kv.half() if case["src"] == "f16" else kv
        st["k"], st["v"] = kv[:, :, :h], kv[:, :, h:]
        st["start"] = _ints(g, 0, cap - n, b)
        st["pos"] = (_ints(g, 0, max(0, case["far"] - n), b)[:, None]
                     + torch.arange(n, device=DEV, dtype=torch.int32)).contiguous()
        st["planes"] = tuple((torch.full((b, cap, h, D // 2), 0x88, dtype=torch.uint8, device=DEV),
                              torch.full((b, cap, h, D // 2), 0x88, dtype=torch.uint8, device=DEV),
                              torch.zeros((b, cap, h), dtype=torch.float16, device=DEV))
                             for _ in range(2))
    elif op == "attend":
        b, h = case["batch"], case["hkv"]
        st = {"q": (_normal(g, b, case["queries"], case["heads"], D) * 1.2).half(),
              "prefix": _cache(g, case["prefix"], h), "own": _cache(g, b, case["cap"], h),
              "lens": _lengths(g, b, case["cap"])}
    elif op == "weights":
        b, n, h, t = case["batch"], case["queries"], case["hkv"], case["tokens"]
        st = {"q": (_normal(g, b, n, case["heads"], D) * 1.2).half()}
        rows = (t, h) if case["shared"] else (b, t, h)
        st["k"] = _pack(_keys(g, *rows))
        st["lens"] = None if case["shared"] else _lengths(g, b, t)
        acc = (h, t) if case["shared"] else (b, h, t)
        st["acc"] = torch.rand(acc, generator=g, device=DEV)
        # the log-sum-exp over these tokens and as much again over others
        s = _scores(case, st, torch.float32)
        st["lse"] = (torch.logsumexp(s, -1) + torch.rand(s.shape[:-1], generator=g, device=DEV))
        st["lse"] = _per_query(case, st["lse"]).float().contiguous()
    else:
        b, h, t = case["batch"], case["hkv"], case["tokens"]
        planes = [[torch.randint(0, 256, (b, t, h, D // 2), generator=g, device=DEV,
                                 dtype=torch.uint8) for _ in range(2)]
                  + [(torch.rand((b, t, h), generator=g, device=DEV) * 0.01).half()]
                  for _ in range(2)]
        # heavy-tailed, and many tokens that nothing has looked at
        acc = torch.exp(3.0 * _normal(g, b, h, t))
        acc = torch.where(acc < 0.1, torch.zeros_like(acc), acc)
        lens = _lengths(g, b, t)
        lens[1::2] = t
        cap = case["keep"] + 16  # with room for the next tokens
        st = {"k": tuple(planes[0]), "v": tuple(planes[1]), "acc": acc, "lens": lens,
              "k_out": tuple(torch.zeros((b, cap) + x.shape[2:], dtype=x.dtype, device=DEV) for x in planes[0]),
              "v_out": tuple(torch.zeros((b, cap) + x.shape[2:], dtype=x.dtype, device=DEV) for x in planes[1]),
              "acc_out": torch.zeros((b, h, cap), device=DEV)}
    return {"case": dict(case), **st}


# ------------------------------------------------------------- plain forms
def _values(mode, hi, lo, scale, dtype=torch.float32):
    """The rows a cache's planes stand for."""
    def nibbles(p):
        return torch.stack([p & 15, p >> 4], -1).flatten(-2).to(dtype) - 8.0
    s = scale.to(dtype)[..., None]
    if mode == 0:
        return nibbles(hi) * s
    return (16.0 * nibbles(hi) + nibbles(lo)) * s / 16.0


def _turned(x, angle, mag, layout, rot):
    """x [..., heads, dim] with its first `rot` values turned by angle [..., rot / 2] (fp64)."""
    c, s = (torch.cos(angle) * mag).float()[..., None, :], (torch.sin(angle) * mag).float()[..., None, :]
    x = x.float()
    if layout == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * c - b * s, a * s + b * c], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _by_head(case, x):
    """[batch, queries, heads, ...] as [batch, hkv, queries, group, ...]."""
    b, n, h = x.shape[:3]
    return x.reshape(b, n, case["hkv"], h // case["hkv"], *x.shape[3:]).transpose(1, 2)


def _per_query(case, x):
    """Rows [(batch,) hkv, queries * group (of all sequences where shared)] as [batch, queries, heads]."""
    b, n, h = case["batch"], case["queries"], case["hkv"]
    if case["shared"]:
        return x.reshape(h, b, n, -1).permute(1, 2, 0, 3).reshape(b, n, -1)
    return x.reshape(b, h, n, -1).transpose(1, 2).reshape(b, n, -1)


def _visible(lens, queries, group, cap):
    """[batch, 1, queries * group, cap]: query i of a sequence sees its tokens up to lens - queries + i."""
    last = lens[:, None].long() - queries + torch.arange(queries, device=DEV)
    ok = torch.arange(cap, device=DEV) <= last[..., None]
    return ok.repeat_interleave(group, 1)[:, None]


def _scores(case, st, dtype):
    """Scores of the queries against the cache of a `weights` case, -inf where hidden."""
    q = _by_head(case, st["q"].to(dtype))  # [b, hkv, n, g, D]
    k = _values(case["mode"], *st["k"], dtype=dtype)
    if case["shared"]:
        rows = q.transpose(0, 1).flatten(1, 3)  # [hkv, b n g, D]
        return rows @ k.permute(1, 2, 0) * RSD
    s = q.flatten(2, 3) @ k.permute(0, 2, 3, 1) * RSD  # [b, hkv, n g, t]
    ok = _visible(st["lens"], case["queries"], case["heads"] // case["hkv"], case["tokens"])
    return torch.where(ok, s, torch.full_like(s, -math.inf))


def _plain_rope(case, st):
    sign = -1.0 if case["inverse"] else 1.0
    angle = st["pos"].double()[:, None] * st["freq"] * sign
    y = _turned(st["x"], angle, st["mag"], case["layout"], case["rot"])
    return y.half() if case["dst"] == "f16" else y


def _plain_append(case, st):
    angle = st["pos"].double()[..., None] * st["freq"]
    k = _turned(st["k"], angle, st["mag"], case["layout"], case["rot"]).half()
    row = st["start"][:, None].long() + torch.arange(case["new"], device=DEV)
    at = torch.arange(case["batch"], device=DEV)[:, None]
    out = []
    for planes, x in zip(st["planes"], (k, st["v"].half())):
        new = _pack(x)
        planes[0][at, row], planes[1][at, row], planes[2][at, row] = new
        out.append(_values(case["mode"], *(p[at, row] for p in planes)).half())
    return out


def _plain_attend(case, st):
    mode, b, n, hkv = case["mode"], case["batch"], case["queries"], case["hkv"]
    group = case["heads"] // hkv
    q = _by_head(case, st["q"].float())  # [b, hkv, n, g, D]
    (kp, vp), (ko, vo) = ([_values(mode, *x) for x in st[c]] for c in ("prefix", "own"))
    sp = q.transpose(0, 1).flatten(1, 3) @ kp.permute(1, 2, 0) * RSD  # [hkv, b n g, P]
    so = q.flatten(2, 3) @ ko.permute(0, 2, 3, 1) * RSD  # [b, hkv, n g, cap]
    ok = _visible(st["lens"], n, group, case["cap"])
    so = torch.where(ok, so, torch.full_like(so, -math.inf))
    most = so.amax(-1)
    if case["prefix"]:
        most = torch.maximum(most, sp.amax(-1).reshape(hkv, b, -1).transpose(0, 1))
    base = torch.where(most == -math.inf, torch.zeros_like(most), most)
    po = torch.exp(so - base[..., None])
    pp = torch.exp(sp - base.transpose(0, 1).reshape(hkv, -1, 1))
    total = po.sum(-1) + pp.sum(-1).reshape(hkv, b, -1).transpose(0, 1)
    o = po @ vo.transpose(1, 2) + (pp @ vp.transpose(0, 1)).reshape(hkv, b, -1, D).transpose(0, 1)
    o = torch.where((total == 0)[..., None], torch.zeros_like(o), o / total[..., None])
    lse = torch.log(total) + base
    o = o.reshape(b, hkv, n, group, D).transpose(1, 2).reshape(b, n, -1, D)
    return o.half(), lse.reshape(b, hkv, n, group).transpose(1, 2).reshape(b, n, -1)


def _plain_weights(case, st):
    s = _scores(case, st, torch.float32)
    lse = _by_head(case, st["lse"])  # [b, hkv, n, g]
    lse = lse.transpose(0, 1).flatten(1) if case["shared"] else lse.flatten(2)
    seen = (s > -math.inf) & (lse > -math.inf)[..., None]
    st["acc"] += torch.where(seen, torch.exp(s - lse[..., None]), torch.zeros_like(s)).sum(-2)
    return st["acc"]


def _plain_evict(case, st):
    b, h, t, keep = case["batch"], case["hkv"], case["tokens"], case["keep"]
    lens = st["lens"].long()
    at = torch.arange(t, device=DEV)
    held = (at < case["sinks"]) | (at >= lens[:, None] - case["recent"])
    key = torch.where(held[:, None], torch.full_like(st["acc"], math.inf), st["acc"])
    key = torch.where((at < lens[:, None])[:, None], key, torch.full_like(key, -math.inf))
    best = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :keep]
    n = lens.clamp(max=keep)
    valid = (torch.arange(keep, device=DEV) < n[:, None])[:, None]
    best = torch.where(valid, best, torch.full_like(best, t)).sort(-1).values
    kept = torch.where(valid, best, torch.full_like(best, -1)).int()
    src = torch.where(valid, best, torch.zeros_like(best)).transpose(1, 2)  # [b, keep, hkv]
    rows = torch.arange(b, device=DEV)[:, None, None], src, torch.arange(h, device=DEV)
    for planes, out in ((st["k"], st["k_out"]), (st["v"], st["v_out"])):
        for x, y in zip(planes, out):
            new = x[rows]
            ok = valid.transpose(1, 2).expand(b, keep, h)
            y[:, :keep] = torch.where(ok[..., None] if x.dim() == 4 else ok, new, y[:, :keep])
    st["acc_out"].zero_()
    acc = torch.gather(st["acc"], 2, src.transpose(1, 2))
    st["acc_out"][..., :keep] = torch.where(valid, acc, torch.zeros_like(acc))
    return st["k_out"], st["v_out"], st["acc_out"], kept, n.int()


# --------------------------------------------------------------- the calls
_LAYOUT = {"half": 0, "pairs": 1}  # ROPE_HALF, ROPE_PAIRS


def _own(case, st):
    import w8_quantized_linear_b200 as bn

    op = case["op"]
    if op == "rope":
        return bn.rope(st["x"], st["pos"], st["phases"], st["mag"], layout=_LAYOUT[case["layout"]],
                       inverse=case["inverse"],
                       dtype=torch.float16 if case["dst"] == "f16" else torch.float32)
    if op == "append":
        bn.kv_append(st["k"], st["v"], st["start"], *st["planes"], pos=st["pos"],
                     phases=st["phases"], magnitude=st["mag"], layout=_LAYOUT[case["layout"]])
        return list(bn.kv_read(case["mode"], st["start"], case["new"], *st["planes"]))
    if op == "attend":
        return bn.prefix_attention(case["mode"], st["q"], st["prefix"], st["own"], st["lens"])
    if op == "weights":
        return bn.kv_weights(case["mode"], st["q"], st["lse"], st["k"], st["acc"], st["lens"])
    kept, lens = bn.kv_evict(st["acc"], st["lens"], case["keep"], case["sinks"], case["recent"],
                             st["k"], st["v"], st["k_out"], st["v_out"], st["acc_out"])
    return st["k_out"], st["v_out"], st["acc_out"], kept, lens


def run(state):
    case = state["case"]
    if own:
        return _own(case, state)
    return {"rope": _plain_rope, "append": _plain_append, "attend": _plain_attend,
            "weights": _plain_weights, "evict": _plain_evict}[case["op"]](case, state)


# --------------------------------------------------------------- the floor
def work(case):
    """Each input read once and each output written once; own tokens at their mean length."""
    op = case["op"]
    size = {"f16": 2, "f32": 4}
    if op == "rope":
        n = case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": n * (size[case["src"]] + size[case["dst"]]) + 4 * case["tokens"]
                + 4 * case["rot"], "flops": 3 * case["tokens"] * case["heads"] * case["rot"]}
    row = D // 2 + 2 if case.get("mode") == 0 else D + 2  # bytes of a cached row that a mode reads
    if op == "append":
        rows = 2 * case["batch"] * case["new"] * case["hkv"]
        return {"bytes": rows * (size[case["src"]] * D + (D + 2) + row + 2 * D)
                + 4 * case["batch"] * (case["new"] + 1), "flops": rows * D * 8}
    if op == "evict":
        b, h, t, keep = case["batch"], case["hkv"], case["tokens"], case["keep"]
        return {"bytes": b * h * (4 * t + keep * (2 * 2 * (D + 2) + 4 + 4)), "flops": 0}
    b, n, heads, hkv = case["batch"], case["queries"], case["heads"], case["hkv"]
    if op == "attend":
        own_tokens = b * case["cap"] // 2
        return {"bytes": 2 * row * hkv * (case["prefix"] + own_tokens) + b * n * heads * (4 * D + 4),
                "flops": 4 * D * n * heads * (b * case["prefix"] + own_tokens)}
    t = case["tokens"] if case["shared"] else b * case["tokens"] // 2
    return {"bytes": hkv * t * (row + 8) + b * n * heads * (2 * D + 4),
            "flops": 2 * D * n * heads * t * (b if case["shared"] else 1)}


# --------------------------------------------------------------- in 64 bits
def _codes(mode, hi, lo, scale):
    """The same rows in 64 bits, from the combined byte."""
    even, odd = ((hi & 15), (hi >> 4)) if mode == 0 else ((hi & 15) * 16 + (lo & 15), (hi >> 4) * 16 + (lo >> 4))
    u = torch.empty(hi.shape[:-1] + (D,), dtype=torch.float64, device=DEV)
    u[..., 0::2], u[..., 1::2] = even.double(), odd.double()
    return (u - 8.0) * scale.double()[..., None] if mode == 0 else (u - 136.0) / 16.0 * scale.double()[..., None]


def _turned_exact(case, x, pos, mag, freq, sign):
    """The rotation as a complex product."""
    r, half = case["rot"], case["rot"] // 2
    x = x.double()
    first = torch.arange(half, device=DEV) if case["layout"] == "half" else torch.arange(0, r, 2, device=DEV)
    second = first + (half if case["layout"] == "half" else 1)
    z = torch.complex(x[..., first], x[..., second])
    turn = pos.double()[..., None, None] * freq * sign
    z = z * torch.polar(torch.full_like(turn, mag), turn)
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "evict":  # choices and copies: no computed numbers
        return None
    if op == "rope":
        return _turned_exact(case, st["x"], st["pos"], st["mag"], st["freq"], -1.0 if case["inverse"] else 1.0)
    if op == "append":
        out = []
        k = _turned_exact(case, st["k"], st["pos"], st["mag"], st["freq"], 1.0)
        for x in (k, st["v"].double()):
            x = x.half().double()
            s = (x.abs().amax(-1, keepdim=True) / 7.0).half().double()
            t = torch.where(s == 0, torch.zeros_like(x), x / torch.where(s == 0, torch.ones_like(s), s))
            q = torch.round(t)
            r = torch.round((t - q) * 16.0).clamp(-8, 7) if case["mode"] else torch.zeros_like(q)
            out.append((q + r / 16.0) * s)
        return out
    mode, hkv = case["mode"], case["hkv"]
    group = case["heads"] // hkv
    q = st["q"].double() / math.sqrt(D)
    if op == "attend":
        (kp, vp), (ko, vo) = ([_codes(mode, *x) for x in st[c]] for c in ("prefix", "own"))
        outs, lses = [], []
        for b, m in enumerate(st["lens"].tolist()):
            k, v = torch.cat([kp, ko[b, :m]]), torch.cat([vp, vo[b, :m]])
            s = torch.einsum("ihgd,thd->ihgt", q[b].unflatten(1, (hkv, group)), k)
            place = torch.arange(k.shape[0], device=DEV) - case["prefix"]
            late = place[None] > m - case["queries"] + torch.arange(case["queries"], device=DEV)[:, None]
            s = s.masked_fill(late[:, None, None] & (place >= 0), -math.inf)
            lse = torch.logsumexp(s, -1)
            p = torch.exp(s - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[..., None])
            outs.append(torch.einsum("ihgt,thd->ihgd", p, v).flatten(1, 2))
            lses.append(lse.flatten(1, 2))
        return torch.stack(outs), torch.stack(lses)
    acc = st["acc"].double()
    lse = st["lse"].double()
    k = _codes(mode, *st["k"])
    for b in range(case["batch"]):
        kb, m = (k, None) if case["shared"] else (k[b], int(st["lens"][b]))
        s = torch.einsum("ihgd,thd->higt", q[b].unflatten(1, (hkv, group)), kb)
        w = torch.exp(s - lse[b].unflatten(1, (hkv, group)).transpose(0, 1)[..., None])
        if case["shared"]:
            acc += w.sum((1, 2))
            continue
        t = torch.arange(case["tokens"], device=DEV)
        late = t[None] > m - case["queries"] + torch.arange(case["queries"], device=DEV)[:, None]
        acc[b] += w.masked_fill(late[None, :, None], 0.0).sum((1, 2))
    return acc
