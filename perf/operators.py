"""The operators of a verify window over a paged key/value cache, as cases to
measure: norms and rotation of queries and keys, the quantising write of the
cache and its reading back, and the attention of drafted tokens over it.

``listed()`` and ``draw()`` give the cases, ``prepare()`` a case's inputs on
the GPU, ``run()`` one pass (the plain form, or with ``own`` the framework's
calls), ``exact()`` the same outputs in 64 bits and ``work()`` the bytes and
operations a pass cannot do without.
"""

import math

import torch

own = False


def _api():
    from confidence_scheduled_speculative_gb300 import api
    return api


# ------------------------------------------------------------------ cases

def listed():
    return [
        # single tokens of four short chats: the smallest call, latency only
        _attend("attend_tokens_tiny", B=4, window=1, lo=16, hi=256, hq=8, hkv=2, D=64, page=16, cache="bf16"),
        # decoding without drafts: 32 requests of up to 8192 tokens, 8-bit cache
        _attend("attend_tokens", B=32, window=1, lo=1, hi=8192, hq=32, hkv=8, D=128, page=64, cache="e4m3"),
        # a verify window of up to 8 drafts a request (32 requests, small pages)
        _attend("attend_window", B=32, window=9, lo=1, hi=8192, hq=32, hkv=8, D=128, page=16, cache="bf16"),
        # the largest batch: 256 requests, up to 16 drafts, 64 query heads
        _attend("attend_window_large", B=256, window=17, lo=1, hi=8192, hq=64, hkv=8, D=128, page=64, cache="bf16"),
        # two long documents with a tree of up to 32 drafted tokens, five query heads a key head
        _attend("attend_tree_long", B=2, window=32, lo=100000, hi=131040, hq=40, hkv=8, D=128, page=64, cache="e4m3", tree=True),
        # the cache write of the smallest window (a handful of rows)
        _append("append_tiny", B=4, window=5, lo=16, hi=256, hq=8, hkv=2, D=64, page=16, cache="bf16"),
        # the write of the largest batch's window, quantised
        _append("append_window", B=256, window=17, lo=1, hi=8192, hq=64, hkv=8, D=128, page=64, cache="e4m3"),
        # eight prompts of up to 4096 tokens enter an empty cache
        _append("append_prompt", B=8, window=4096, lo=0, hi=0, hq=32, hkv=8, D=128, page=64, cache="bf16"),
        # a draft model's small fp32 heads, part of each rotated, neighbouring pairs
        _rope("rope_draft", B=4, window=5, lo=16, hi=256, hq=12, hkv=4, D=80, rope=64, interleaved=True, dtype="f32"),
        # queries and keys of four prompts, no cache
        _rope("rope_prompt", B=4, window=4096, lo=0, hi=0, hq=64, hkv=8, D=128, rope=128, interleaved=False, dtype="bf16"),
        # one short prefix read back in 32 bits
        _read("read_short", B=1, lo=0, hi=301, hkv=2, D=64, page=16, cache="bf16", out="f32"),
        # the prefixes of 32 requests leave an 8-bit cache
        _read("read_prefixes", B=32, lo=0, hi=8192, hkv=8, D=128, page=64, cache="e4m3", out="bf16"),
    ]


def _attend(name, B, window, lo, hi, hq, hkv, D, page, cache, tree=False):
    return {"name": name, "op": "attend", "B": B, "window": window, "lo": lo, "hi": hi, "hq": hq,
            "hkv": hkv, "D": D, "page": page, "cache": cache, "tree": tree}


def _append(name, B, window, lo, hi, hq, hkv, D, page, cache):
    return {"name": name, "op": "append", "B": B, "window": window, "lo": lo, "hi": hi, "hq": hq,
            "hkv": hkv, "D": D, "rope": D, "interleaved": False, "page": page, "cache": cache,
            "dtype": "bf16"}


def _rope(name, B, window, lo, hi, hq, hkv, D, rope, interleaved, dtype):
    return {"name": name, "op": "rope", "B": B, "window": window, "lo": lo, "hi": hi, "hq": hq,
            "hkv": hkv, "D": D, "rope": rope, "interleaved": interleaved, "dtype": dtype}


def _read(name, B, lo, hi, hkv, D, page, cache, out):
    return {"name": name, "op": "read", "B": B, "window": 0, "lo": lo, "hi": hi, "hkv": hkv, "D": D,
            "page": page, "cache": cache, "out": out}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the listed ones' ranges."""
    largest = {}
    for c in listed():
        w = work(c)
        for k in ("bytes", "flops"):
            largest[c["op"], k] = max(largest.get((c["op"], k), 0), w[k])
    while True:
        op = rng.choice(["attend", "attend", "append", "rope", "read"])
        hkv = rng.choice([1, 2, 3, 4, 8])
        hq = hkv * rng.choice([1, 2, 3, 4, 5, 7, 8])
        D = rng.choice([64, 128])
        page = rng.choice([16, 32, 64, 128])
        cache = rng.choice(["bf16", "e4m3"])
        if op == "attend":
            B, hi = _log(rng, 1, 256), _log(rng, 8, 131040)
            c = _attend("", B, _log(rng, 1, 32), rng.randrange(0, hi), hi, hq, hkv, D, page, cache,
                        rng.random() < 0.5)
            # the plain form holds every score and a 32-bit copy of the cache
            if B * hi * hkv * D > 256 * 8192 * 1024 or B * hi * hq * c["window"] > 256 * 8192 * 17 * 64:
                continue
        elif op == "append":
            hi = _log(rng, 8, 8192)
            c = _append("", _log(rng, 1, 256), _log(rng, 1, 4096), rng.randrange(0, hi), hi, hq, hkv,
                        D, page, cache)
        elif op == "rope":
            D = rng.choice([64, 80, 96, 128, 256])
            hi = _log(rng, 8, 8192)
            c = _rope("", _log(rng, 1, 256), _log(rng, 1, 4096), rng.randrange(0, hi), hi, hq, hkv, D,
                      rng.choice([D, D // 2]), rng.random() < 0.5, rng.choice(["bf16", "f32"]))
        else:
            hi = _log(rng, 8, 131072)
            c = _read("", _log(rng, 1, 64), rng.randrange(0, hi), hi, hkv, D, page, cache,
                      rng.choice(["bf16", "f32"]))
        w = work(c)
        if all(w[k] <= largest[op, k] for k in w):
            del c["name"]
            return c


# ---------------------------------------------------------------- lengths
# The lengths of a case are spread evenly over its range and dealt to the
# requests by the seed, so the work is the same for every seed.

def _prefixes(c):
    return [c["lo"] + (c["hi"] - c["lo"]) * (i + 1) // c["B"] for i in range(c["B"])]


def _windows(c):
    return [-(-c["window"] * (i + 1) // c["B"]) for i in range(c["B"])]


def _pairs(c):
    """(prefix, window) of each request before the seed deals them: long and
    short prefixes meet long and short windows."""
    p, w = _prefixes(c), _windows(c)
    step = 1 + 2 * (c["B"] // 3)
    while math.gcd(step, c["B"]) != 1:
        step += 1
    return [(p[i], w[i * step % c["B"]]) for i in range(c["B"])]


_BYTES = {"bf16": 2, "f32": 4, "e4m3": 1}


def work(case):
    c = case
    pairs = _pairs(c)
    rows = sum(w for _, w in pairs)
    slot = 2 * c["hkv"] * (c["D"] * _BYTES[c.get("cache", "bf16")] + (4 if c.get("cache") == "e4m3" else 0))
    if c["op"] == "attend":
        tokens = sum(p + w for p, w in pairs)
        seen = sum(p * w + (w * (w + 1) // 2 if not c["tree"] else w * min(w, 4)) for p, w in pairs)
        return {"bytes": tokens * slot + rows * c["hq"] * (c["D"] * 4 + 4), "flops": 4 * c["D"] * c["hq"] * seen}
    e = _BYTES[c.get("dtype", "bf16")]
    if c["op"] == "read":
        tokens = sum(p for p, _ in pairs)
        out = 2 * c["hkv"] * c["D"] * _BYTES[c["out"]]
        return {"bytes": tokens * (slot + out), "flops": tokens * 2 * c["hkv"] * c["D"]}
    angles = min(rows, c["hi"] + c["window"]) * c["rope"] * 4
    q_k = rows * (c["hq"] + c["hkv"]) * c["D"]
    if c["op"] == "rope":
        return {"bytes": 2 * q_k * e + angles, "flops": 10 * q_k}
    return {"bytes": q_k * e + rows * c["hkv"] * c["D"] * e + rows * c["hq"] * c["D"] * e + rows * slot + angles,
            "flops": 10 * q_k + 4 * rows * c["hkv"] * c["D"]}


# ----------------------------------------------------------------- inputs

_DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


def _randn(gen, shape, dtype, scale=1.0):
    if dtype == torch.float32:
        return torch.randn(shape, generator=gen, device="cuda") * scale
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16) * scale


def _quantised(x):
    """Codes and scales of x [..., D]: the state that an earlier write left."""
    x = x.float()
    s = (x.abs().amax(-1) / 448).clamp(min=2.0 ** -100)
    return (x / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn), s


def _make_cache(c, gen, tokens, filled):
    """A pool of pages and the requests' page tables; `tokens` [B] are the
    positions each request needs. With `filled`, every page holds what an
    earlier step wrote (another request's tokens past a request's own)."""
    page, hkv, D = c["page"], c["hkv"], c["D"]
    need = [-(-t // page) for t in tokens]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    width = max(need) + 1
    at = torch.tensor([0] + need, device="cuda").cumsum(0)[:-1]
    col = torch.arange(width, device="cuda")
    table = order[(at[:, None] + col[None, :]).clamp(max=n_pages - 1)].contiguous()
    kind = c["cache"]
    shape = (n_pages, page, hkv, D)
    cache = {"table": table}
    for n in ("k", "v"):
        if not filled:
            cache[n] = torch.zeros(shape, device="cuda", dtype=torch.bfloat16).to(_DTYPE[kind])
            if kind == "e4m3":
                cache[n + "_scale"] = torch.zeros((n_pages, hkv, page), device="cuda")
        elif kind == "bf16":
            cache[n] = _randn(gen, shape, torch.bfloat16)
        else:
            cache[n] = torch.empty(shape, device="cuda", dtype=torch.float8_e4m3fn)
            cache[n + "_scale"] = torch.empty((n_pages, hkv, page), device="cuda")
            for i in range(0, n_pages, 1024):  # in pieces: the 32-bit values are four times the codes
                codes, s = _quantised(_randn(gen, (min(1024, n_pages - i),) + shape[1:], torch.bfloat16))
                cache[n][i:i + 1024] = codes
                cache[n + "_scale"][i:i + 1024] = s.transpose(1, 2)
    return cache


def _angles(n, rope):
    """cos and sin of position * 10000^(-2i/rope): what a model keeps."""
    f = 10000.0 ** (-torch.arange(0, rope, 2, device="cuda", dtype=torch.float64) / rope)
    a = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def _tree(rng_cpu, w):
    """Ancestor bits and depths of a random tree of w drafted tokens."""
    bits, depth = [1], [0]
    for i in range(1, w):
        p = int(torch.randint(max(0, i - 4), i, (1,), generator=rng_cpu))
        bits.append(bits[p] | 1 << i)
        depth.append(depth[p] + 1)
    return [b - (1 << 32) if b >> 31 else b for b in bits], depth


def prepare(case, seed):
    c = case
    gen = torch.Generator("cuda").manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    pairs = _pairs(c)
    pairs = [pairs[i] for i in torch.randperm(c["B"], generator=cpu).tolist()]
    prefix, win = [p for p, _ in pairs], [w for _, w in pairs]
    i32 = dict(dtype=torch.int32, device="cuda")
    s = {"case": c, "rows": sum(win), "prefix": torch.tensor(prefix, **i32),
         "cu": torch.tensor([0] + win, device="cuda").cumsum(0).to(torch.int32),
         "status": torch.zeros(1, **i32)}
    if c["op"] == "read":
        s["cache"] = _make_cache(c, gen, prefix, True)
        s["start"] = torch.zeros(c["B"], **i32)
        s["cu"] = torch.tensor([0] + prefix, device="cuda").cumsum(0).to(torch.int32)
        s["rows"] = sum(prefix)
        s["k_out"] = torch.zeros((s["rows"], c["hkv"], c["D"]), device="cuda", dtype=_DTYPE[c["out"]])
        s["v_out"] = torch.zeros_like(s["k_out"])
        if own:
            _handle(s)
        return s
    # the window is padded to a multiple of 64 rows, as a captured step is
    rows = s["rows"]
    cap = -(-rows // 64) * 64
    req = torch.repeat_interleave(torch.arange(c["B"], device="cuda"),
                                  torch.tensor(win, device="cuda")).to(torch.int32)
    j = torch.arange(rows, **i32) - s["cu"][req.long()]
    pad = cap - rows
    s["req"] = torch.cat([req, torch.full((pad,), -1, **i32)])
    s["pos"] = torch.cat([s["prefix"][req.long()] + j, torch.zeros(pad, **i32)])
    s["totals"] = torch.tensor([rows, cap], **i32)
    hq, hkv, D = c["hq"], c["hkv"], c["D"]
    if c["op"] == "attend":
        s["cache"] = _make_cache(c, gen, [p + w for p, w in pairs], True)
        s["q"] = _randn(gen, (cap, hq, D), torch.bfloat16, 2.0)  # scores of a few units: some heads are peaked
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros((cap, hq), device="cuda")
        s["scale"] = D ** -0.5
        s["tree"] = None
        if c["tree"]:
            bits = [b for w in win for b in _tree(cpu, w)[0]]
            s["tree"] = torch.tensor(bits + [0] * pad, **i32)
    else:
        dt = _DTYPE[c["dtype"]]
        # one projection's output: queries, keys and values of a row side by side
        qkv = _randn(gen, (cap, hq + 2 * hkv, D), dt, 1.5)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["q_weight"] = (1 + 0.1 * torch.randn(D, generator=gen, device="cuda")).to(dt)
        s["k_weight"] = (1 + 0.1 * torch.randn(D, generator=gen, device="cuda")).to(dt)
        s["eps"] = 1e-6
        s["cos_sin"] = _angles(c["hi"] + c["window"] + 1, c["rope"])
        s["q_out"] = torch.zeros((cap, hq, D), device="cuda", dtype=dt)
        if c["op"] == "append":
            s["cache"] = _make_cache(c, gen, [p + w for p, w in pairs], False)
        else:
            s["k_out"] = torch.zeros((cap, hkv, D), device="cuda", dtype=dt)
    if own and "cache" in s:
        _handle(s)
    return s


def _handle(s):
    """What a program keeps with its cache: the framework's descriptor of it
    and a workspace."""
    api, k = _api(), s["cache"]
    s["kv"] = api.KVCache(k["k"], k["v"], k["table"], k.get("k_scale"), k.get("v_scale"))
    if s["case"]["op"] == "attend":
        s["ws"] = api.workspace(api.dspark_tree_attention_workspace_bytes(s["case"]["hq"], s["case"]["D"]))


# ------------------------------------------------------------- plain form

def _norm_rope(x, w, eps, cos_sin, pos, rope, interleaved):
    x = x.float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.float()
    t = cos_sin[pos.long()][:, None, :]
    cos, sin = t[..., :rope // 2], t[..., rope // 2:]
    r, rest = y[..., :rope], y[..., rope:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., :rope // 2], r[..., rope // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, rest], -1)


def _gather(c, cache, n, width):
    """Values [B, width, hkv, D] in 32 bits of the positions 0..width-1."""
    pages = cache["table"][:, :-(-width // c["page"])].long()
    if c["cache"] == "e4m3":
        x = cache[n].view(torch.uint8)[pages].view(torch.float8_e4m3fn).float()
        x = x * cache[n + "_scale"][pages].transpose(2, 3)[..., None]
    else:
        x = cache[n][pages].float()
    return x.flatten(1, 2)[:, :width]


def _plain_attend(s):
    c = s["case"]
    B, W, hq, hkv, D, rows = c["B"], c["window"], c["hq"], c["hkv"], c["D"], s["rows"]
    S, G = c["hi"] + W, hq // hkv
    req = s["req"][:rows].long()
    j = torch.arange(rows, device="cuda") - s["cu"][req].long()
    q = torch.zeros((B, W, hq, D), device="cuda")
    q[req, j] = s["q"][:rows].float()
    k = _gather(c, s["cache"], "k", S).permute(0, 2, 3, 1)
    x = torch.matmul(q.view(B, W, hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, hkv, W * G, D), k)
    del k
    x = x.mul_(s["scale"]).view(B, hkv, W, G, S)
    p = torch.arange(S, device="cuda") - s["prefix"].long()[:, None]  # place in the window, negative before it
    at = torch.arange(W, device="cuda")
    if s["tree"] is None:
        sees = p[:, None, :] <= at[None, :, None]
    else:
        bits = torch.zeros((B, W), device="cuda", dtype=torch.int64)
        bits[req, j] = s["tree"][:rows].long()
        sees = (p < 0)[:, None, :] | ((p < 32)[:, None, :]
                                      & ((bits[:, :, None] >> p.clamp(0, 31)[:, None, :]) & 1).bool())
    x.masked_fill_(~sees[:, None, :, None, :], float("-inf"))
    m = x.amax(-1, keepdim=True)
    m0 = m.masked_fill(m == float("-inf"), 0.0)
    x.sub_(m0).exp_()
    l = x.sum(-1, keepdim=True)
    v = _gather(c, s["cache"], "v", S).permute(0, 2, 1, 3)
    o = torch.matmul(x.view(B, hkv, W * G, S), v).view(B, hkv, W, G, D)
    o = torch.where(l > 0, o / l, 0.0)
    lse = (m0 + l.log()).squeeze(-1)
    out, out_lse = torch.zeros_like(s["out"]), torch.zeros_like(s["lse"])
    out[:rows] = o.permute(0, 2, 1, 3, 4).reshape(B, W, hq, D)[req, j].to(out.dtype)
    out_lse[:rows] = lse.permute(0, 2, 1, 3).reshape(B, W, hq)[req, j]
    return {"out": out, "lse": out_lse}


def _plain_rope(s):
    c, rows = s["case"], s["rows"]
    q_out, k_out = torch.zeros_like(s["q_out"]), torch.zeros_like(s["k_out"])
    for_pos = s["pos"][:rows]
    a = (s["eps"], s["cos_sin"], for_pos, c["rope"], c["interleaved"])
    q_out[:rows] = _norm_rope(s["q"][:rows], s["q_weight"], *a).to(q_out.dtype)
    k_out[:rows] = _norm_rope(s["k"][:rows], s["k_weight"], *a).to(k_out.dtype)
    return {"q": q_out, "k": k_out}


def _plain_append(s):
    c, rows, cache = s["case"], s["rows"], s["cache"]
    req, pos = s["req"][:rows].long(), s["pos"][:rows].long()
    a = (s["eps"], s["cos_sin"], pos, c["rope"], c["interleaved"])
    q_out = torch.zeros_like(s["q_out"])
    q_out[:rows] = _norm_rope(s["q"][:rows], s["q_weight"], *a).to(q_out.dtype)
    k = _norm_rope(s["k"][:rows], s["k_weight"], *a)
    page, slot = cache["table"][req, pos // c["page"]].long(), pos % c["page"]
    _store(c, cache, "k", k, page, slot)
    _store(c, cache, "v", s["v"][:rows].float(), page, slot)
    return _appended(s, q_out)


def _store(c, cache, n, x, page, slot):
    if c["cache"] == "bf16":
        cache[n][page, slot] = x.to(torch.bfloat16)
        return
    codes, scale = _quantised(x)
    cache[n].view(torch.uint8)[page, slot] = codes.view(torch.uint8)
    cache[n + "_scale"].transpose(1, 2)[page, slot] = scale


def _appended(s, q_out):
    got = {"q": q_out}
    got.update({n: t for n, t in s["cache"].items() if n != "table"})
    return got


def _plain_read(s):
    c = s["case"]
    req = torch.repeat_interleave(torch.arange(c["B"], device="cuda"), s["cu"].long().diff(),
                                  output_size=s["rows"])
    pos = s["start"].long()[req] + torch.arange(s["rows"], device="cuda") - s["cu"].long()[req]
    page, slot = s["cache"]["table"][req, pos // c["page"]].long(), pos % c["page"]
    return {n: _load(c, s["cache"], n, page, slot).to(s["k_out"].dtype) for n in ("k", "v")}


def _load(c, cache, n, page, slot):
    if c["cache"] == "bf16":
        return cache[n][page, slot].float()
    codes = cache[n].view(torch.uint8)[page, slot].view(torch.float8_e4m3fn).float()
    return codes * cache[n + "_scale"].transpose(1, 2)[page, slot][..., None]


# -------------------------------------------------------------------- run

def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"attend": _plain_attend, "append": _plain_append, "rope": _plain_rope,
                "read": _plain_read}[op](s)
    api, c = _api(), s["case"]
    if op == "attend":
        api.dspark_tree_attention(s["q"], s["kv"], cu_seqlens=s["cu"], prefix_lens=s["prefix"],
                                  scale=s["scale"], out=s["out"], lse=s["lse"], ancestors=s["tree"],
                                  workspace=s["ws"], status=s["status"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "read":
        api.dspark_kv_read(s["kv"], start=s["start"], cu_rows=s["cu"], k_out=s["k_out"],
                           v_out=s["v_out"], status=s["status"])
        return {"k": s["k_out"], "v": s["v_out"]}
    common = dict(pos=s["pos"], totals=s["totals"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                  eps=s["eps"], cos_sin=s["cos_sin"], interleaved=c["interleaved"],
                  q_out=s["q_out"], status=s["status"])
    if op == "append":
        api.dspark_kv_append(s["k"], s["v"], s["kv"], q=s["q"], req=s["req"], **common)
        return _appended(s, s["q_out"])
    api.dspark_qk_norm_rope(s["q"], s["k"], k_out=s["k_out"], **common)
    return {"q": s["q_out"], "k": s["k_out"]}


# ------------------------------------------------------- 64-bit definition

def exact(case, seed):
    s = prepare(case, seed)
    c, rows = case, s["rows"]
    f64 = torch.float64
    cu = s["cu"].tolist()
    prefix = s["prefix"].tolist()

    def cached(n, r, lo, hi):
        """Positions lo..hi-1 of request r: [hi-lo, hkv, D] in 64 bits."""
        p = torch.arange(lo, hi, device="cuda")
        page, slot = s["cache"]["table"][r][p // c["page"]].long(), p % c["page"]
        if c["cache"] != "e4m3":
            return s["cache"][n][page, slot].to(f64)
        code = s["cache"][n].view(torch.uint8)[page, slot].to(torch.int32)
        e, f = code >> 3 & 15, (code & 7).to(f64)
        mag = torch.where(e > 0, (1 + f / 8) * torch.exp2(e.to(f64) - 7), f / 8 * 2.0 ** -6)
        x = torch.where(code > 127, -mag, mag)
        return x * s["cache"][n + "_scale"][page, :, slot].to(f64)[..., None]

    if c["op"] == "read":
        got = {n: torch.zeros(s["k_out"].shape, device="cuda", dtype=f64) for n in ("k", "v")}
        for n in got:
            for r in range(c["B"]):
                if cu[r + 1] > cu[r]:
                    got[n][cu[r]:cu[r + 1]] = cached(n, r, 0, cu[r + 1] - cu[r])
        return got

    if c["op"] == "attend":
        out = torch.zeros(s["out"].shape, device="cuda", dtype=f64)
        lse = torch.zeros(s["lse"].shape, device="cuda", dtype=f64)
        G = c["hq"] // c["hkv"]
        for r in range(c["B"]):
            lo, hi, P = cu[r], cu[r + 1], prefix[r]
            L, n = hi - lo, P + hi - lo
            hidden = torch.zeros((L, n), dtype=torch.bool)
            for i in range(L):
                bits = (1 << i + 1) - 1 if s["tree"] is None else int(s["tree"][lo + i])
                for t in range(L):
                    hidden[i, P + t] = not bits >> t & 1
            hidden = hidden.cuda()
            k, v = cached("k", r, 0, n), cached("v", r, 0, n)
            for h in range(c["hq"]):
                z = s["q"][lo:hi, h].to(f64) @ k[:, h // G].T * s["scale"]
                z[hidden] = float("-inf")
                total = torch.logsumexp(z, 1)
                lse[lo:hi, h] = total
                out[lo:hi, h] = torch.exp(z - total[:, None]) @ v[:, h // G]
        return {"out": out, "lse": lse}

    def turned(x, w):
        x = x[:rows].to(f64)
        y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * w.to(f64)
        R = c["rope"]
        z = s["cos_sin"].to(f64)[s["pos"][:rows].long()]
        z = torch.complex(z[:, :R // 2], z[:, R // 2:])[:, None]
        even = torch.arange(0, R, 2, device="cuda") if c["interleaved"] else torch.arange(R // 2, device="cuda")
        odd = even + (1 if c["interleaved"] else R // 2)
        t = torch.complex(y[..., even], y[..., odd]) * z
        y[..., even], y[..., odd] = t.real, t.imag
        return y

    def padded(x, like):
        full = torch.zeros(like.shape, device="cuda", dtype=f64)
        full[:rows] = x
        return full

    q, k = turned(s["q"], s["q_weight"]), turned(s["k"], s["k_weight"])
    got = {"q": padded(q, s["q_out"])}
    if c["op"] == "rope":
        got["k"] = padded(k, s["k_out"])
        return got
    for n, x in (("k", k), ("v", s["v"][:rows].to(f64))):
        pool = torch.zeros(s["cache"][n].shape, device="cuda", dtype=f64)
        p = s["pos"][:rows].long()
        page, slot = s["cache"]["table"][s["req"][:rows].long(), p // c["page"]].long(), p % c["page"]
        if c["cache"] == "e4m3":
            scale = x.abs().amax(-1) / 448
            x = x / scale[..., None]
            step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
            x = torch.round(x / step) * step
            scales = torch.zeros(s["cache"][n + "_scale"].shape, device="cuda", dtype=f64)
            scales[page, :, slot] = scale
            got[n + "_scale"] = scales
        pool[page, slot] = x
        got[n] = pool
    return got
