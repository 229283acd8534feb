"""The operators of a latent cache and of a cache that is kept short, as cases to
measure: the write of latent rows, attention over them in the absorbed form (a window of
drafted tokens) and in the expanded one (a prompt), the attention weights that a cache's
positions gather, and the eviction of those that gathered little.

``listed()`` and ``draw()`` give the cases, ``prepare()`` a case's inputs on
the GPU, ``run()`` one pass (the plain form, or with ``own`` the framework's
calls), ``exact()`` the same outputs in 64 bits and ``work()`` the bytes and
operations a pass cannot do without.
"""

import math

import torch

own = False

LATENT, ROPE = 512, 64  # a token's latent vector, and the part of its key that is rotated
NOPE, VALUE = 128, 128  # a head's expanded key without that part, and its expanded value


def _api():
    from confidence_scheduled_speculative_gb300 import api
    return api


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the latent rows of a handful of drafted tokens: the smallest write, latency only
        _append("latent_append_tiny", B=4, window=5, lo=16, hi=256, hq=16, page=16),
        # the largest batch's window, the rotated parts of all 128 heads' queries with it
        _append("latent_append_window", B=256, window=17, lo=1, hi=8192, hq=128, page=64),
        # single tokens of four short chats, an eighth of the heads: latency
        _latent("latent_tokens_tiny", B=4, window=1, lo=16, hi=256, hq=16, page=16),
        # decoding without drafts, all heads: 32 requests of up to 8192 tokens
        _latent("latent_tokens", B=32, window=1, lo=1, hi=8192, hq=128, page=64),
        # a verify window of up to 8 drafts a request, an eighth of the heads, small pages
        _latent("latent_window", B=32, window=9, lo=1, hi=8192, hq=16, page=16),
        # two long documents with a tree of up to 32 drafted tokens
        _latent("latent_tree_long", B=2, window=32, lo=100000, hi=131040, hq=64, page=64, tree=True),
        # four short prompts, expanded
        _prompt("prompt_short", B=4, window=128, lo=0, hi=0, hq=16),
        # the second part of two long prompts behind their first parts
        _prompt("prompt_long", B=2, window=8192, lo=2000, hi=4000, hq=32),
        # what single tokens attend to, over 8-bit keys
        _weights("weights_tokens", B=32, window=1, lo=1, hi=8192, hq=32, hkv=8, D=128, page=64, cache="e4m3"),
        # what the accepted tokens of verify windows attend to
        _weights("weights_window", B=32, window=9, lo=1, hi=8192, hq=32, hkv=8, D=128, page=16, cache="bf16"),
        # each step of a long generation: a window's tokens more than the cache is to keep
        _evict("evict_step", B=32, lo=4096, hi=4113, keep=4096, recent=1024, hkv=8, D=128, page=64, cache="bf16"),
        # long prompts cut down to an eighth before decoding begins
        _evict("evict_prompts", B=4, lo=60000, hi=131040, keep=16384, recent=4096, hkv=8, D=128, page=64,
               cache="e4m3"),
    ]


def _append(name, B, window, lo, hi, hq, page, interleaved=True):
    return {"name": name, "op": "append", "B": B, "window": window, "lo": lo, "hi": hi, "hq": hq,
            "page": page, "interleaved": interleaved}


def _latent(name, B, window, lo, hi, hq, page, tree=False):
    return {"name": name, "op": "latent", "B": B, "window": window, "lo": lo, "hi": hi, "hq": hq,
            "page": page, "tree": tree}


def _prompt(name, B, window, lo, hi, hq):
    return {"name": name, "op": "prompt", "B": B, "window": window, "lo": lo, "hi": hi, "hq": hq}


def _weights(name, B, window, lo, hi, hq, hkv, D, page, cache):
    return {"name": name, "op": "weights", "B": B, "window": window, "lo": lo, "hi": hi, "hq": hq,
            "hkv": hkv, "D": D, "page": page, "cache": cache}


def _evict(name, B, lo, hi, keep, recent, hkv, D, page, cache):
    return {"name": name, "op": "evict", "B": B, "window": 0, "lo": lo, "hi": hi, "keep": keep,
            "recent": recent, "hkv": hkv, "D": D, "page": page, "cache": cache}


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
        op = rng.choice(["latent", "latent", "append", "prompt", "weights", "evict"])
        heads = rng.choice([1, 2, 5, 8, 16, 20, 32, 64, 128])
        hkv = rng.choice([1, 2, 3, 4, 8])
        hq = hkv * rng.choice([1, 2, 3, 4, 5, 7, 8])
        page = rng.choice([16, 32, 64, 128])
        D, cache = rng.choice([64, 128]), rng.choice(["bf16", "e4m3"])
        if op == "append":
            hi = _log(rng, 8, 8192)
            c = _append("", _log(rng, 1, 256), _log(rng, 1, 4096), rng.randrange(0, hi), hi, heads, page,
                        rng.random() < 0.5)
        elif op == "latent":
            B, hi = _log(rng, 1, 128), _log(rng, 8, 131040)
            c = _latent("", B, _log(rng, 1, 32), rng.randrange(0, hi), hi, heads, page, rng.random() < 0.5)
            # the plain form holds every score and a 32-bit copy of the cache
            if B * hi * heads * c["window"] > 2 * 131072 * 32 * 64 or B * hi > 64 * 8192:
                continue
        elif op == "prompt":
            hi = _log(rng, 8, 8192) if rng.random() < 0.5 else 0
            c = _prompt("", _log(rng, 1, 16), _log(rng, 1, 8192), rng.randrange(0, hi + 1), hi, heads)
            if heads * c["window"] * (c["window"] + hi) > 32 * 8192 * 12288:
                continue
        elif op == "weights":
            B, hi = _log(rng, 1, 256), _log(rng, 8, 131040)
            c = _weights("", B, _log(rng, 1, 32), rng.randrange(0, hi), hi, hq, hkv, D, page, cache)
            if B * hi * hkv * D > 64 * 8192 * 1024 or B * hi * hq * c["window"] > 32 * 8192 * 32 * 32:
                continue
        else:
            hi = _log(rng, 8, 131040)
            keep = _log(rng, 1, hi)
            c = _evict("", _log(rng, 1, 64), rng.randrange(0, hi), hi, keep, rng.randrange(0, keep + 1),
                       hkv, D, page, cache)
            if c["B"] * hi * hkv * D > 32 * 8192 * 8 * 128:
                continue
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


def _seen(c, pairs):
    """(row, position) pairs that a query head looks at."""
    return sum(p * w + (w * min(w, 4) if c.get("tree") else w * (w + 1) // 2) for p, w in pairs)


_BYTES = {"bf16": 2, "e4m3": 1}


def work(case):
    c = case
    pairs = _pairs(c)
    rows, tokens = sum(w for _, w in pairs), sum(p + w for p, w in pairs)
    if c["op"] == "append":
        row, turned = (LATENT + ROPE) * 2, rows * c["hq"] * ROPE * 2
        return {"bytes": 2 * rows * row + 2 * turned + min(rows, c["hi"] + c["window"]) * ROPE * 4,
                "flops": rows * (4 * LATENT + 3 * ROPE * (1 + c["hq"]))}
    if c["op"] == "latent":
        return {"bytes": tokens * (LATENT + ROPE) * 2 + rows * c["hq"] * ((2 * LATENT + ROPE) * 2 + 4),
                "flops": 2 * (2 * LATENT + ROPE) * c["hq"] * _seen(c, pairs)}
    if c["op"] == "prompt":
        return {"bytes": rows * c["hq"] * ((NOPE + ROPE + VALUE) * 2 + 4)
                + tokens * (c["hq"] * (NOPE + VALUE) + ROPE) * 2,
                "flops": 2 * (NOPE + ROPE + VALUE) * c["hq"] * _seen(c, pairs)}
    key = c["D"] * _BYTES[c["cache"]] + (4 if c["cache"] == "e4m3" else 0)
    if c["op"] == "weights":
        return {"bytes": tokens * c["hkv"] * (key + 8) + rows * c["hq"] * (c["D"] * 2 + 4),
                "flops": 2 * c["D"] * c["hq"] * _seen(c, pairs)}
    moved = kept = 0
    for n in _prefixes(c):
        k, r = min(c["keep"], n), min(c["recent"], n)
        kept += k
        if n > k:  # of the others, each is as likely to be kept
            behind = n - k
            moved += min(r, behind) + max(behind - r, 0) * (k - r) // max(n - r, 1)
    return {"bytes": c["hkv"] * ((tokens + kept) * 8 + moved * 4 * key), "flops": tokens * c["hkv"]}


# ----------------------------------------------------------------- inputs

_DTYPE = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
_I32 = dict(dtype=torch.int32, device="cuda")


def _randn(gen, shape, scale=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16) * scale


def _quantised(x):
    """Codes and scales of x [..., D]: the state that an earlier write left."""
    x = x.float()
    s = (x.abs().amax(-1) / 448).clamp(min=2.0 ** -100)
    return (x / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn), s


def _table(c, gen, tokens):
    """The requests' page tables over a pool; `tokens` [B] are the positions
    each request needs."""
    need = [-(-t // c["page"]) for t in tokens]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    at = torch.tensor([0] + need, device="cuda").cumsum(0)[:-1]
    col = torch.arange(max(need) + 1, device="cuda")
    return n_pages, order[(at[:, None] + col[None, :]).clamp(max=n_pages - 1)].contiguous()


def _kv_cache(c, gen, tokens):
    """Keys and values of an earlier step in every page (another request's
    tokens past a request's own)."""
    page, hkv, D = c["page"], c["hkv"], c["D"]
    n_pages, table = _table(c, gen, tokens)
    shape, cache = (n_pages, page, hkv, D), {"table": table}
    for n in ("k", "v"):
        if c["cache"] == "bf16":
            cache[n] = _randn(gen, shape)
        else:
            cache[n] = torch.empty(shape, device="cuda", dtype=torch.float8_e4m3fn)
            cache[n + "_scale"] = torch.empty((n_pages, hkv, page), device="cuda")
            for i in range(0, n_pages, 1024):  # in pieces: the 32-bit values are four times the codes
                codes, s = _quantised(_randn(gen, (min(1024, n_pages - i),) + shape[1:]))
                cache[n][i:i + 1024] = codes
                cache[n + "_scale"][i:i + 1024] = s.transpose(1, 2)
    return cache


def _angles(n):
    """cos and sin of position * 10000^(-2i/ROPE): what a model keeps."""
    f = 10000.0 ** (-torch.arange(0, ROPE, 2, device="cuda", dtype=torch.float64) / ROPE)
    a = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def _tree(rng_cpu, w):
    """Ancestor bits of a random tree of w drafted tokens."""
    bits = [1]
    for i in range(1, w):
        p = int(torch.randint(max(0, i - 4), i, (1,), generator=rng_cpu))
        bits.append(bits[p] | 1 << i)
    return [b - (1 << 32) if b >> 31 else b for b in bits]


def prepare(case, seed):
    c = case
    gen = torch.Generator("cuda").manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    pairs = _pairs(c)
    pairs = [pairs[i] for i in torch.randperm(c["B"], generator=cpu).tolist()]
    prefix, win = [p for p, _ in pairs], [w for _, w in pairs]
    s = {"case": c, "rows": sum(win), "prefix": torch.tensor(prefix, **_I32),
         "cu": torch.tensor([0] + win, device="cuda").cumsum(0).to(torch.int32),
         "status": torch.zeros(1, **_I32)}
    if c["op"] == "evict":
        _prepare_evict(s, gen, prefix)
    elif c["op"] == "prompt":
        _prepare_prompt(s, gen, pairs)
    else:
        _prepare_window(s, gen, cpu, prefix, win)
    if own:
        _handle(s)
    return s


def _prepare_window(s, gen, cpu, prefix, win):
    c, rows = s["case"], s["rows"]
    # the window is padded to a multiple of 64 rows, as a captured step is
    cap = -(-rows // 64) * 64
    pad = cap - rows
    req = torch.repeat_interleave(torch.arange(c["B"], device="cuda"),
                                  torch.tensor(win, device="cuda")).to(torch.int32)
    j = torch.arange(rows, **_I32) - s["cu"][req.long()]
    s["req"] = torch.cat([req, torch.full((pad,), -1, **_I32)])
    s["pos"] = torch.cat([s["prefix"][req.long()] + j, torch.zeros(pad, **_I32)])
    s["totals"] = torch.tensor([rows, cap], **_I32)
    tokens = [p + w for p, w in zip(prefix, win)]
    hq = c["hq"]
    if c["op"] == "append":
        # what the two down projections leave: a latent vector and a key part a token, and
        # queries of which the last ROPE elements are to be rotated
        s["rows_in"] = _randn(gen, (cap, LATENT + ROPE), 1.5)
        s["q"] = _randn(gen, (cap, hq, NOPE + ROPE), 1.5)
        s["weight"] = (1 + 0.1 * torch.randn(LATENT, generator=gen, device="cuda")).bfloat16()
        s["eps"] = 1e-6
        s["cos_sin"] = _angles(c["hi"] + c["window"] + 1)
        # where the absorbed queries go: the rotated part behind the latent one
        s["q_latent"] = torch.zeros((cap, hq, LATENT + ROPE), device="cuda", dtype=torch.bfloat16)
        n_pages, s["table"] = _table(c, gen, tokens)
        s["pages"] = torch.zeros((n_pages, c["page"], LATENT + ROPE), device="cuda", dtype=torch.bfloat16)
    elif c["op"] == "latent":
        n_pages, s["table"] = _table(c, gen, tokens)
        s["pages"] = _randn(gen, (n_pages, c["page"], LATENT + ROPE))
        s["q"] = _randn(gen, (cap, hq, LATENT + ROPE), 2.0)  # scores of a few units: some heads are peaked
        s["scale"] = (LATENT + ROPE) ** -0.5
        s["out"] = torch.zeros((cap, hq, LATENT), device="cuda", dtype=torch.bfloat16)
        s["lse"] = torch.zeros((cap, hq), device="cuda")
        s["tree"] = None
        if c["tree"]:
            s["tree"] = torch.tensor([b for w in win for b in _tree(cpu, w)] + [0] * pad, **_I32)
    else:
        s["cache"] = _kv_cache(c, gen, tokens)
        s["q"] = _randn(gen, (cap, hq, c["D"]), 2.0)
        s["scale"] = c["D"] ** -0.5
        S = c["hi"] + c["window"]
        # what earlier steps gathered, the positions of the entries, the tokens accepted
        s["weights"] = torch.rand((c["B"], c["hkv"], S), generator=gen, device="cuda")
        s["weights_out"] = torch.zeros_like(s["weights"])
        s["positions"] = torch.arange(S, **_I32).expand(c["B"], c["hkv"], S).contiguous()
        s["counts"] = torch.tensor([1 + (7 * i) % w for i, w in enumerate(win)], **_I32)
        s["decay"] = 0.98
        s["lse"] = torch.zeros((cap, hq), device="cuda")
        _attended_lse(s)


def _prepare_prompt(s, gen, pairs):
    c, rows, hq = s["case"], s["rows"], s["case"]["hq"]
    lens = [p + w for p, w in pairs]
    tokens = sum(lens)
    s["cu_k"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    s["q"] = _randn(gen, (rows, hq, NOPE + ROPE), 2.0)
    # one up projection's output: a head's keys and values side by side
    kv = _randn(gen, (tokens, hq, NOPE + VALUE))
    s["k"], s["v"] = kv[..., :NOPE], kv[..., NOPE:]
    s["k_shared"] = _randn(gen, (tokens, ROPE))
    s["scale"] = (NOPE + ROPE) ** -0.5
    s["out"] = torch.zeros((rows, hq, VALUE), device="cuda", dtype=torch.bfloat16)
    s["lse"] = torch.zeros((rows, hq), device="cuda")


def _prepare_evict(s, gen, lens):
    c = s["case"]
    S = max(lens)
    s["lens"] = s["prefix"]
    s["cache"] = _kv_cache(c, gen, lens)
    shape = (c["B"], c["hkv"], S)
    # gathered weights: a few positions have most, some of the newest none yet
    w = torch.exp(2 * torch.randn(shape, generator=gen, device="cuda"))
    s["weights"] = torch.where(torch.rand(shape, generator=gen, device="cuda") < 0.1, 0.0, w)
    # entries of earlier evictions lie in no order, the newest at the end
    n = s["lens"].long()[:, None, None]
    slot = torch.arange(S, device="cuda").expand(shape)
    mixed = torch.rand(shape, generator=gen, device="cuda").masked_fill(slot >= n - c["recent"], 2.0)
    s["positions"] = torch.argsort(torch.argsort(mixed, dim=-1, stable=True), dim=-1).to(torch.int32)
    s["now"] = s["lens"].clone()
    s["weights_out"], s["positions_out"] = torch.zeros_like(s["weights"]), torch.zeros_like(s["positions"])
    s["new_lens"] = torch.zeros(c["B"], **_I32)


def _handle(s):
    """What a program keeps with its cache: the framework's descriptor of it
    and a workspace."""
    api, c = _api(), s["case"]
    if "pages" in s:
        s["lc"] = api.LatentCache(s["pages"], s["table"], LATENT)
    if "cache" in s:
        k = s["cache"]
        s["kv"] = api.KVCache(k["k"], k["v"], k["table"], k.get("k_scale"), k.get("v_scale"))
    if c["op"] == "latent":
        s["ws"] = api.workspace(api.dspark_latent_attention_workspace_bytes(c["hq"], LATENT))
    elif c["op"] == "evict":
        s["ws"] = api.workspace(api.dspark_kv_evict_workspace_bytes(c["B"], c["hkv"], s["weights"].size(2)))


# ------------------------------------------------------------- plain form

def _turned(x, cos_sin, pos, interleaved):
    """The pairs of x [rows, heads, ROPE] rotated, in 32 bits."""
    x, t = x.float(), cos_sin[pos.long()][:, None, :]
    cos, sin = t[..., :ROPE // 2], t[..., ROPE // 2:]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    a, b = x[..., :ROPE // 2], x[..., ROPE // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_append(s):
    c, rows = s["case"], s["rows"]
    pos, req = s["pos"][:rows], s["req"][:rows].long()
    q_latent = s["q_latent"]
    q_latent[:rows, :, LATENT:] = _turned(s["q"][:rows, :, NOPE:], s["cos_sin"], pos, c["interleaved"])
    x = s["rows_in"][:rows, :LATENT].float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * s["weight"].float()
    r = _turned(s["rows_in"][:rows, None, LATENT:], s["cos_sin"], pos, c["interleaved"])[:, 0]
    page, slot = s["table"][req, (pos // c["page"]).long()].long(), (pos % c["page"]).long()
    s["pages"][page, slot] = torch.cat([x, r], -1).bfloat16()
    return {"pages": s["pages"], "q": q_latent}


def _window_bits(s, W):
    """Whether token i of request r's window sees token j: [B, W, W]."""
    c, rows = s["case"], s["rows"]
    at = torch.arange(W, device="cuda")
    if s.get("tree") is None:
        return (at[None, :] <= at[:, None]).expand(c["B"], W, W)
    req = s["req"][:rows].long()
    bits = torch.zeros((c["B"], W), device="cuda", dtype=torch.int64)
    bits[req, torch.arange(rows, device="cuda") - s["cu"].long()[req]] = s["tree"][:rows].long()
    return (bits[:, :, None] >> at & 1).bool()


def _window_sees(s, S):
    """Whether token i of request r's window sees position p: [B, W, S]."""
    W = s["case"]["window"]
    p = torch.arange(S, device="cuda") - s["prefix"].long()[:, None]  # place in the window
    inside = _window_bits(s, W).gather(2, p.clamp(0, W - 1)[:, None, :].expand(-1, W, -1))
    return (p < 0)[:, None, :] | ((p < W)[:, None, :] & inside)


def _padded(s, x):
    """Rows [rows, ...] as [B, W, ...] in 32 bits, zeros where a request has fewer."""
    c, rows = s["case"], s["rows"]
    req = s["req"][:rows].long()
    full = torch.zeros((c["B"], c["window"]) + x.shape[1:], device="cuda")
    full[req, torch.arange(rows, device="cuda") - s["cu"].long()[req]] = x[:rows].float()
    return full


def _unpadded(s, x, like):
    rows = s["rows"]
    req = s["req"][:rows].long()
    out = torch.zeros_like(like)
    out[:rows] = x[req, torch.arange(rows, device="cuda") - s["cu"].long()[req]].to(out.dtype)
    return out


def _plain_latent(s):
    c = s["case"]
    B, W, hq = c["B"], c["window"], c["hq"]
    S = c["hi"] + W
    kv = s["pages"][s["table"][:, :-(-S // c["page"])].long()].flatten(1, 2)[:, :S].float()
    x = torch.matmul(_padded(s, s["q"]).view(B, W * hq, LATENT + ROPE), kv.transpose(1, 2))
    x = x.mul_(s["scale"]).view(B, W, hq, S)
    x.masked_fill_(~_window_sees(s, S)[:, :, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    m = m.masked_fill_(m == float("-inf"), 0.0)
    x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, W * hq, S), kv[..., :LATENT]).view(B, W, hq, LATENT)
    o = torch.where(l > 0, o / l, 0.0)
    return {"out": _unpadded(s, o, s["out"]), "lse": _unpadded(s, (m + l.log()).squeeze(-1), s["lse"])}


def _plain_prompt(s):
    out, lse = torch.empty_like(s["out"]), torch.empty_like(s["lse"])
    cu, cu_k = s["cu"].tolist(), s["cu_k"].tolist()
    for r in range(s["case"]["B"]):
        q0, q1, k0, k1 = cu[r], cu[r + 1], cu_k[r], cu_k[r + 1]
        q = s["q"][q0:q1].float().transpose(0, 1)
        x = torch.matmul(q[..., :NOPE], s["k"][k0:k1].float().permute(1, 2, 0))
        x += torch.matmul(q[..., NOPE:], s["k_shared"][k0:k1].float().t())
        x.mul_(s["scale"])
        row, col = torch.arange(q1 - q0, device="cuda"), torch.arange(k1 - k0, device="cuda")
        x.masked_fill_(col[None, :] > row[:, None] + (k1 - k0) - (q1 - q0), float("-inf"))
        m = x.amax(-1, keepdim=True)
        x.sub_(m).exp_()
        l = x.sum(-1, keepdim=True)
        o = torch.matmul(x, s["v"][k0:k1].float().transpose(0, 1)) / l
        out[q0:q1] = o.transpose(0, 1).to(out.dtype)
        lse[q0:q1] = (m + l.log()).squeeze(-1).t()
    return {"out": out, "lse": lse}


def _scores(s):
    """Scores of the window's rows over the cache, those unseen -inf: [B, hkv, W, G, S]."""
    c, cache = s["case"], s["cache"]
    B, W, hkv, D, G = c["B"], c["window"], c["hkv"], c["D"], c["hq"] // c["hkv"]
    S = c["hi"] + W
    pages = cache["table"][:, :-(-S // c["page"])].long()
    if c["cache"] == "e4m3":
        k = cache["k"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).float()
        k = k * cache["k_scale"][pages].transpose(2, 3)[..., None]
    else:
        k = cache["k"][pages].float()
    k = k.flatten(1, 2)[:, :S].permute(0, 2, 3, 1)
    q = _padded(s, s["q"]).view(B, W, hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, hkv, W * G, D)
    x = torch.matmul(q, k).mul_(s["scale"]).view(B, hkv, W, G, S)
    return x.masked_fill_(~_window_sees(s, S)[:, None, :, None, :], float("-inf"))


def _attended_lse(s):
    """What the attention before left: each row's log of its sum of exponentials."""
    c = s["case"]
    x = torch.logsumexp(_scores(s), -1)
    s["lse"].copy_(_unpadded(s, x.permute(0, 2, 1, 3).reshape(c["B"], c["window"], c["hq"]), s["lse"]))


def _plain_weights(s):
    c = s["case"]
    B, W, hkv, G = c["B"], c["window"], c["hkv"], c["hq"] // c["hkv"]
    lse = _padded(s, s["lse"]).view(B, W, hkv, G).permute(0, 2, 1, 3)
    at = torch.arange(W, device="cuda")
    x = _scores(s).sub_(lse[..., None]).exp_()
    x.masked_fill_((at >= s["counts"][:, None])[:, None, :, None, None], 0.0)
    x = x.sum((2, 3))
    P, n = s["prefix"].long()[:, None, None], (s["prefix"] + s["counts"]).long()[:, None, None]
    p = torch.arange(x.size(-1), device="cuda")
    old, pos = s["weights"], s["positions"]
    return {"weights": torch.where(p < P, old * s["decay"] + x, torch.where(p < n, x, 0.0)),
            "positions": torch.where((p >= P) & (p < n), p.to(torch.int32), pos)}


def _plain_evict(s):
    c, cache = s["case"], s["cache"]
    S, keep = s["weights"].size(2), c["keep"]
    n = s["lens"].long()[:, None, None]
    slot = torch.arange(S, device="cuda")
    fresh = s["positions"] >= (s["now"] - c["recent"])[:, None, None]
    key = torch.where(fresh, float("inf"), s["weights"]).masked_fill(slot >= n, -1.0)
    order = torch.argsort(key, dim=-1, descending=True, stable=True)
    stays = torch.zeros(key.shape, device="cuda", dtype=torch.bool).scatter_(-1, order[..., :keep], True)
    stays &= slot < n
    new = n.clamp(max=keep)
    # the entries that stay from behind the new end, in order, into the places left before it
    to, of = (~stays & (slot < new)).nonzero(as_tuple=True), (stays & (slot >= new)).nonzero(as_tuple=True)
    weights, positions = s["weights"].clone(), s["positions"].clone()
    for t in (weights, positions):
        t[to] = t[of]
        t.masked_fill_(slot >= new, 0)
    page = [cache["table"].long()[r, p // c["page"]] for r, _, p in (to, of)]
    tok = [p % c["page"] for _, _, p in (to, of)]
    for name in ("k", "v"):
        x = cache[name].view(torch.uint8) if c["cache"] == "e4m3" else cache[name]
        x[page[0], tok[0], to[1]] = x[page[1], tok[1], of[1]]
        if c["cache"] == "e4m3":
            x = cache[name + "_scale"]
            x[page[0], to[1], tok[0]] = x[page[1], of[1], tok[1]]
    return _evicted(s, new[:, 0, 0].to(torch.int32), weights, positions)


def _evicted(s, lens, weights, positions):
    got = {"lens": lens, "weights": weights, "positions": positions}
    got.update({n: t for n, t in s["cache"].items() if n != "table"})
    return got


# -------------------------------------------------------------------- run

def run(state):
    s = state
    c = s["case"]
    if not own:
        return {"append": _plain_append, "latent": _plain_latent, "prompt": _plain_prompt,
                "weights": _plain_weights, "evict": _plain_evict}[c["op"]](s)
    api = _api()
    if c["op"] == "append":
        api.dspark_latent_append(s["rows_in"], s["lc"], req=s["req"], pos=s["pos"], totals=s["totals"],
                                 q_rope=s["q"][..., NOPE:], q_rope_out=s["q_latent"][..., LATENT:],
                                 weight=s["weight"], eps=s["eps"], cos_sin=s["cos_sin"],
                                 interleaved=c["interleaved"], status=s["status"])
        return {"pages": s["pages"], "q": s["q_latent"]}
    if c["op"] == "latent":
        api.dspark_latent_attention(s["q"], s["lc"], cu_seqlens=s["cu"], prefix_lens=s["prefix"],
                                    scale=s["scale"], out=s["out"], lse=s["lse"], ancestors=s["tree"],
                                    workspace=s["ws"], status=s["status"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "prompt":
        api.dspark_prompt_attention(s["q"], s["k"], s["v"], k_shared=s["k_shared"], cu_seqlens=s["cu"],
                                    cu_keys=s["cu_k"], scale=s["scale"], out=s["out"], lse=s["lse"],
                                    status=s["status"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "weights":
        api.dspark_attention_weights(s["q"], s["kv"], lse=s["lse"], cu_seqlens=s["cu"],
                                     prefix_lens=s["prefix"], scale=s["scale"], counts=s["counts"],
                                     decay=s["decay"], weights=s["weights"], weights_out=s["weights_out"],
                                     pos=s["pos"], positions=s["positions"], status=s["status"])
        return {"weights": s["weights_out"], "positions": s["positions"]}
    api.dspark_kv_evict(s["kv"], lens=s["lens"], now=s["now"], keep=c["keep"], recent=c["recent"],
                        weights=s["weights"], weights_out=s["weights_out"], positions=s["positions"],
                        positions_out=s["positions_out"], new_lens=s["new_lens"], workspace=s["ws"],
                        status=s["status"])
    return _evicted(s, s["new_lens"], s["weights_out"], s["positions_out"])


# ------------------------------------------------------- 64-bit definition

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "latent": _exact_latent, "prompt": _exact_prompt,
            "weights": _exact_weights, "evict": _exact_evict}[case["op"]](s)


_F64 = torch.float64


def _zeros(shape):
    return torch.zeros(shape, device="cuda", dtype=_F64)


def _exact_append(s):
    c, rows = s["case"], s["rows"]
    p = s["pos"][:rows].long()
    z = torch.complex(*s["cos_sin"].to(_F64)[p].split(ROPE // 2, 1))[:, None]
    a = torch.arange(0, ROPE, 2) if c["interleaved"] else torch.arange(ROPE // 2)
    b = a + (1 if c["interleaved"] else ROPE // 2)

    def turn(x):
        x = x.to(_F64)
        t = torch.complex(x[..., a], x[..., b]) * z
        y = torch.empty_like(x)
        y[..., a], y[..., b] = t.real, t.imag
        return y

    q = _zeros(s["q_latent"].shape)
    q[:rows, :, LATENT:] = turn(s["q"][:rows, :, NOPE:])
    x = s["rows_in"][:rows, :LATENT].to(_F64)
    x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * s["weight"].to(_F64)
    pages = _zeros(s["pages"].shape)
    page = s["table"][s["req"][:rows].long(), p // c["page"]].long()
    pages[page, p % c["page"], :LATENT] = x
    pages[page, p % c["page"], LATENT:] = turn(s["rows_in"][:rows, None, LATENT:])[:, 0]
    return {"pages": pages, "q": q}


def _hidden(s, r, P, L):
    """Which positions of P + L a window's tokens do not see: [L, P + L]."""
    hidden = torch.zeros((L, P + L), dtype=torch.bool)
    lo = int(s["cu"][r])
    for i in range(L):
        bits = (2 << i) - 1 if s.get("tree") is None else int(s["tree"][lo + i])
        for t in range(L):
            hidden[i, P + t] = not bits >> t & 1
    return hidden.cuda()


def _exact_latent(s):
    c, cu, prefix = s["case"], s["cu"].tolist(), s["prefix"].tolist()
    out, lse = _zeros(s["out"].shape), _zeros(s["lse"].shape)
    for r in range(c["B"]):
        lo, hi, P = cu[r], cu[r + 1], prefix[r]
        p = torch.arange(P + hi - lo, device="cuda")
        kv = s["pages"][s["table"][r][p // c["page"]].long(), p % c["page"]].to(_F64)
        hidden = _hidden(s, r, P, hi - lo)
        for h in range(c["hq"]):
            z = s["q"][lo:hi, h].to(_F64) @ kv.T * s["scale"]
            z[hidden] = float("-inf")
            lse[lo:hi, h] = torch.logsumexp(z, 1)
            out[lo:hi, h] = torch.exp(z - lse[lo:hi, h, None]) @ kv[:, :LATENT]
    return {"out": out, "lse": lse}


def _exact_prompt(s):
    c, cu, cu_k = s["case"], s["cu"].tolist(), s["cu_k"].tolist()
    out, lse = _zeros(s["out"].shape), _zeros(s["lse"].shape)
    for r in range(c["B"]):
        lo, hi, k0, k1 = cu[r], cu[r + 1], cu_k[r], cu_k[r + 1]
        for h in range(c["hq"]):
            k = torch.cat([s["k"][k0:k1, h], s["k_shared"][k0:k1]], 1).to(_F64)
            z = s["q"][lo:hi, h].to(_F64) @ k.T * s["scale"]
            z[torch.ones_like(z, dtype=torch.bool).triu((k1 - k0) - (hi - lo) + 1)] = float("-inf")
            lse[lo:hi, h] = torch.logsumexp(z, 1)
            out[lo:hi, h] = torch.exp(z - lse[lo:hi, h, None]) @ s["v"][k0:k1, h].to(_F64)
    return {"out": out, "lse": lse}


def _values64(c, cache, name, page, tok):
    """Entries in 64 bits, as [..., hkv, D]."""
    if c["cache"] != "e4m3":
        return cache[name][page, tok].to(_F64)
    code = cache[name].view(torch.uint8)[page, tok].to(torch.int32)
    e, f = code >> 3 & 15, (code & 7).to(_F64)
    mag = torch.where(e > 0, (1 + f / 8) * torch.exp2(e.to(_F64) - 7), f / 8 * 2.0 ** -6)
    return torch.where(code > 127, -mag, mag) * cache[name + "_scale"][page, :, tok].to(_F64)[..., None]


def _exact_weights(s):
    c, cu, prefix, counts = s["case"], s["cu"].tolist(), s["prefix"].tolist(), s["counts"].tolist()
    weights, positions = _zeros(s["weights"].shape), s["positions"].clone()
    G = c["hq"] // c["hkv"]
    for r in range(c["B"]):
        lo, L, P = cu[r], counts[r], prefix[r]
        p = torch.arange(P + L, device="cuda")
        k = _values64(c, s["cache"], "k", s["cache"]["table"][r][p // c["page"]].long(), p % c["page"])
        hidden = _hidden(s, r, P, L)
        weights[r, :, :P] = s["weights"][r, :, :P].to(_F64) * s["decay"]
        for h in range(c["hq"]):
            z = s["q"][lo:lo + L, h].to(_F64) @ k[:, h // G].T * s["scale"] - s["lse"][lo:lo + L, h, None].to(_F64)
            z[hidden] = float("-inf")
            weights[r, h // G, :P + L] += torch.exp(z).sum(0)
        positions[r, :, P:P + L] = torch.arange(P, P + L, **_I32)
    return {"weights": weights, "positions": positions}


def _exact_evict(s):
    c, keep = s["case"], s["case"]["keep"]
    lens, now = s["lens"].tolist(), s["now"].tolist()
    weights, positions = _zeros(s["weights"].shape), torch.zeros_like(s["positions"])
    got = {n: t.clone() for n, t in s["cache"].items() if n != "table"}
    for r in range(c["B"]):
        n = lens[r]
        new = min(n, keep)
        for h in range(c["hkv"]):
            w, p = s["weights"][r, h, :n].to(_F64), s["positions"][r, h, :n]
            rank = torch.where(p >= now[r] - c["recent"], float("inf"), w)
            best = torch.sort(rank, descending=True, stable=True).indices[:new]
            lies = torch.arange(new, device="cuda")
            behind = best[best >= new].sort().values
            free = torch.ones(new, dtype=torch.bool, device="cuda")
            free[best[best < new]] = False
            free = lies[free]
            lies[free] = behind
            weights[r, h, :new], positions[r, h, :new] = w[lies], p[lies]
            a, b = (s["cache"]["table"][r][x // c["page"]].long() for x in (free, behind))
            for name in got:
                if name.endswith("scale"):
                    got[name][a, h, free % c["page"]] = s["cache"][name][b, h, behind % c["page"]]
                else:
                    x, y = (t.view(torch.uint8) if c["cache"] == "e4m3" else t for t in (got[name], s["cache"][name]))
                    x[a, free % c["page"], h] = y[b, behind % c["page"], h]
    got.update(lens=s["lens"].clamp(max=keep), weights=weights, positions=positions)
    return got
