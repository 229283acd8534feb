"""Plain 64-bit definitions of the latent cache's and the short cache's operators, and
the random problems their tests run on (test infrastructure only).  The rounding bounds
are worked out as in window_oracle."""

import math

import torch

import window_oracle as wo

LATENT, ROPE = 512, 64


class Latent:
    """A random paged latent cache, as window_oracle.attention takes one: one key head
    of [c | r], its value c."""

    def __init__(self, gen, kind, tokens, page, latent=LATENT, rope=ROPE, filled=True, spare=2, pool=None,
                 wide=0, scale=1.0):
        self.kind, self.page, self.latent, self.rope, self.heads = kind, page, latent, rope, 1
        need = [-(-t // page) for t in tokens]
        self.n_pages = pool or sum(need) + spare
        order = torch.randperm(self.n_pages, generator=gen)[:sum(need)].to(torch.int32)
        self.table = torch.full((len(tokens), max(need + [1])), -1, dtype=torch.int32)  # unused: no page
        at = 0
        for r, n in enumerate(need):
            self.table[r, :n] = order[at:at + n]
            at += n
        self.table = self.table.cuda()
        # `wide`: entries beside other columns
        self.pool = torch.zeros((self.n_pages, page, latent + rope + wide), device="cuda", dtype=wo.DTYPES[kind])
        self.pages = self.pool[..., :latent + rope]
        if filled:
            g = torch.Generator("cuda").manual_seed(int(torch.randint(1 << 30, (1,), generator=gen)))
            self.pool.normal_(0, scale, generator=g)

    def lc(self):
        from confidence_scheduled_speculative_gb300 import api
        return api.LatentCache(self.pages, self.table, self.latent)

    def entries(self, r, lo, hi):
        p = torch.arange(lo, hi, device="cuda")
        return self.pages[self.table[r][p // self.page].long(), p % self.page]

    def values(self, which, r, lo, hi):
        x = self.entries(r, lo, hi).double()
        return (x if which == "k" else x[:, :self.latent])[:, None]

    def put(self, r, p, value, part=slice(None)):
        self.pages[int(self.table[r, p // self.page]), p % self.page, part] = value


# ------------------------------------------------------------------ prompts

def prompt(q, k, k_shared, v, scale):
    """q [n, hq, K + S], k [m, hkv, K], k_shared [m, S] or None, v [m, hkv, V]: out, lse
    and the largest errors of 32-bit sums, and sum |weight v|, in 64 bits."""
    n, hq, D = q.shape
    m, hkv = k.shape[:2]
    kk, vv = (t.double().repeat_interleave(hq // hkv, 1).permute(1, 0, 2) for t in (k, v))
    if k_shared is not None:
        kk = torch.cat([kk, k_shared.double().expand(hq, m, -1)], 2)
    qq = q.double().permute(1, 0, 2)
    sees = (torch.arange(m, device="cuda")[None] <= torch.arange(n, device="cuda")[:, None] + m - n)[None]
    z = (qq @ kk.transpose(1, 2) * scale).masked_fill(~sees, -math.inf)
    mx = z.amax(-1, keepdim=True) if m else torch.full((hq, n, 1), -math.inf, device="cuda").double()
    m0 = mx.masked_fill(mx == -math.inf, 0.0)
    w = torch.where(sees, torch.exp(z - m0), 0.0)
    total = w.sum(-1, keepdim=True)
    w = torch.where(total > 0, w / total, 0.0)
    w = torch.where(torch.isnan(total), total, w)
    if bool(torch.isfinite(vv).all()):
        o, o_abs = w @ vv, w @ vv.abs()
    else:  # what a row does not see is left out, not multiplied by zero
        terms = [torch.where(sees[0, i][None, :, None], w[:, i, :, None] * vv, 0.0) for i in range(n)]
        o, o_abs = (torch.stack([f(t).sum(1) for t in terms], 1) for f in (torch.Tensor.clone, torch.abs))
    lse = (m0 + total.log()).squeeze(-1)
    s_abs = (qq.abs() @ torch.nan_to_num(kk, 0, 0, 0).abs().transpose(1, 2)).amax(-1, keepdim=True) * abs(scale) \
        if m else torch.zeros((hq, n, 1), device="cuda").double()
    s_tol = (D + 4) * wo.U32 * s_abs + 16 * wo.U32
    tol = o_abs * (2 * s_tol + 2 * (m + 16) * wo.U32)
    lse_tol = s_tol.squeeze(-1) + (m + 16) * wo.U32 + 4 * wo.U32 * lse.abs()
    return (o.permute(1, 0, 2), lse.permute(1, 0), tol.permute(1, 0, 2), lse_tol.permute(1, 0),
            o_abs.permute(1, 0, 2))


def compare(got, got_lse, want, weight_unit, dtype, tag):
    """Asserts an attention's output rows against their definition (`want`: what prompt or
    window_oracle.attention give); weight_unit: the rounding of a weight."""
    o, lse, tol, lse_tol, o_abs = want
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(o)), tag
    assert torch.equal(torch.isinf(got), torch.isinf(o)), tag
    fine = torch.isfinite(o)
    bound = (tol + weight_unit * o_abs) * (1 + wo.BF16) + wo.out_unit(dtype) * o.abs() + 1e-38
    off = ((got - o).abs() - bound)[fine]
    assert not off.numel() or float(off.max()) <= 0, (tag, float(off.max()))
    if got_lse is None:
        return
    got_lse = got_lse.double()
    assert torch.equal(got_lse == -math.inf, lse == -math.inf), tag
    assert torch.equal(torch.isnan(got_lse), torch.isnan(lse)), tag
    fine = torch.isfinite(lse)
    off = ((got_lse - lse).abs() - lse_tol)[fine]
    assert not off.numel() or float(off.max()) <= 0, (tag, float(off.max()))


# ------------------------------------------------------- gathered weights

def gathered(q, lse, cache, r, P, L, n, bits, scale):
    """What the first n of L rows q [L, hq, D] give each position below P + n, and the
    largest error: [hkv, P + n] each, in 64 bits."""
    hq, D = q.size(1), q.size(2)
    G = hq // cache.heads
    k = cache.values("k", r, 0, P + n).permute(1, 0, 2).repeat_interleave(G, 0)
    qq = q[:n].double().permute(1, 0, 2)
    sees = torch.ones((n, P + n), dtype=torch.bool)
    for i in range(n):
        for t in range(n):
            sees[i, P + t] = bool(bits[i] >> t & 1)
    sees = sees.cuda()[None]
    x = qq @ k.transpose(1, 2) * scale - lse[:n].double().t()[:, :, None]
    e = torch.where(sees, torch.exp(x), 0.0)
    # a score: D products in 32 bits; its difference from lse and that difference to base
    # 2 round once each; the exponential is off by two units, a sum of N terms by N
    s_abs = qq.abs() @ torch.nan_to_num(k, 0, 0, 0).abs().transpose(1, 2) * abs(scale)
    x_tol = (D + 4) * wo.U32 * s_abs + 4 * wo.U32 * (x.abs() + 1) + 4 * wo.U32
    N = n * G
    e_tol = torch.where(sees, e * (x_tol + N * wo.U32), 0.0)

    def fold(t):
        if not n:
            return torch.zeros((cache.heads, P), device="cuda").double()
        return t.view(cache.heads, G, n, P + n).sum((1, 2))

    return fold(e), fold(e_tol)


# ---------------------------------------------------------------- eviction

def evicted(weights, positions, n, now, keep, recent):
    """Of one head's entries (lists): which place each of the new places is filled from."""
    if n <= keep:
        return list(range(n))

    def rank(p):
        fresh = positions[p] >= now - recent
        w = weights[p]
        return (not fresh, 0.0 if fresh else (math.inf if math.isnan(w) else -w), not fresh and math.isnan(w), p)

    stay = sorted(sorted(range(n), key=rank)[:keep])
    behind = [p for p in stay if p >= keep]
    kept = set(stay)
    return [p if p in kept else behind.pop(0) for p in range(keep)]
