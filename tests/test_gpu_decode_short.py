"""Caches that are kept short, as the decode loop uses the calls: append, attend, gather,
evict and go on."""

import math

import numpy as np
import pytest
import torch

import latent_oracle as lo
import window_oracle as wo
from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def decode():
    require_gpu()
    from confidence_scheduled_speculative_gb300 import decode
    return decode


def entries(cache, r, n):
    """Keys and values of request r's first n places in 64 bits: [n, heads, D]."""
    p = torch.arange(n, device="cuda")
    page, tok = cache.block_table[r][p // cache.k.size(1)].long(), p % cache.k.size(1)
    out = []
    for t, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        if s is None:
            out.append(t[page, tok].double())
        else:
            out.append(wo.e4m3_values(t.view(torch.uint8)[page, tok]) * s[page, :, tok].double()[..., None])
    return out


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
def test_rounds_of_eviction(decode, kind):
    """Three windows with an eviction behind each: every place holds the entry of the token
    that the ledger says, those kept are the fresh and the heaviest, and the next window's
    attention is the formula over exactly these entries."""
    B, hq, hkv, D, keep, recent = 3, 8, 2, 64, 24, 8
    dt = torch.float32 if kind == "f32" else torch.bfloat16
    cache = decode.PagedCache(B, 96, hq, hkv, D, page_size=16, dtype=wo.DTYPES[kind], seed=2, ledger=True)
    g = torch.Generator("cuda").manual_seed(5)
    status, lens, now = torch.zeros(1, **I32), torch.zeros(B, **I32), torch.zeros(B, **I32)
    held = {}  # (request, position): the entry as it was stored
    for step, (win, take) in enumerate([([32, 20, 5], [32, 20, 5]), ([9, 17, 6], [4, 17, 1]), ([7, 1, 8], [7, 1, 8]),
                                        ([3, 3, 3], [3, 3, 3])]):
        rows, counts = sum(win), torch.tensor(take, **I32)
        cu = torch.tensor([0] + win, device="cuda").cumsum(0).int()
        req = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(win, device="cuda")).int()
        offset = torch.arange(rows, **I32) - cu[req.long()]
        pos, place = now[req.long()] + offset, lens[req.long()] + offset
        x = torch.randn((rows, hq + 2 * hkv, D), generator=g, device="cuda").to(dt)
        q, k, v = x[:, :hq] * 2, x[:, hq:hq + hkv], x[:, hq + hkv:]
        cache.append(q, k, v, req=req, pos=pos, cache_pos=place, status=status)
        out, lse = torch.zeros((rows, hq, D), device="cuda", dtype=dt), torch.zeros((rows, hq), device="cuda")
        kw = dict(cu_seqlens=cu, prefix_lens=lens.clone(), scale=D ** -0.5, status=status)
        cache.attend(q, out, lse=lse, **kw)
        n = lens.tolist()

        class Held:  # window_oracle's view of the cache
            heads = hkv

            def values(self, which, r, a, b):
                return entries(cache, r, b)[0 if which == "k" else 1][a:b]

        at = 0
        unit = {"bf16": wo.BF16, "e4m3": wo.F16, "f32": 0.0}[kind]
        for r, L in enumerate(win):
            want = wo.attention(q[at:at + L], Held(), r, n[r], L, wo.chain_bits(L), D ** -0.5)
            lo.compare(out[at:at + L], lse[at:at + L], want, unit, dt, (step, r))
            ks, vs = entries(cache, r, n[r] + take[r])
            for i in range(take[r]):
                held[r, int(now[r]) + i] = ks[n[r] + i], vs[n[r] + i]
            at += L
        weights = cache.weights.clone()
        cache.gather(q, lse, pos=pos, counts=counts, decay=0.5, **kw)
        at = 0
        for r, L in enumerate(win):
            e, tol = lo.gathered(q[at:at + L], lse[at:at + L], Held(), r, n[r], L, take[r], wo.chain_bits(L), D ** -0.5)
            e[:, :n[r]] += 0.5 * weights[r, :, :n[r]].double()
            got = cache.weights[r, :, :n[r] + take[r]].double()
            assert bool(((got - e).abs() <= tol + 3 * wo.U32 * e.abs()).all()), (step, r)
            at += L
        lens += counts
        now += counts
        weights, positions, before = cache.weights.clone(), cache.positions.clone(), lens.clone()
        cache.evict(lens=before, now=now, keep=keep, recent=recent, new_lens=lens, status=status)
        assert lens.tolist() == before.clamp(max=keep).tolist()
        for r in range(B):
            m = int(lens[r])
            ks, vs = entries(cache, r, m)
            for h in range(hkv):
                of = lo.evicted(weights[r, h].tolist(), positions[r, h].tolist(), int(before[r]), int(now[r]), keep,
                                recent)
                assert cache.positions[r, h, :m].tolist() == [int(positions[r, h, p]) for p in of]
                assert torch.equal(cache.weights[r, h, :m], weights[r, h][torch.tensor(of, device="cuda")])
                assert set(range(max(int(now[r]) - recent, 0), int(now[r]))) <= set(cache.positions[r, h, :m].tolist())
                for s, p in enumerate(cache.positions[r, h, :m].tolist()):
                    assert torch.equal(ks[s, h], held[r, p][0][h]) and torch.equal(vs[s, h], held[r, p][1][h])
    assert int(status) == 0 and lens.tolist() == [keep, keep, min(17, keep)] and not math.isnan(float(out.sum()))


def test_a_cache_that_keeps_everything(decode):
    """With room for all tokens nothing is evicted, and the loop commits what it does
    without a ledger; cut short, it still runs."""
    def run(keep, recent=16):
        cfg = decode.ToyConfig(keep=keep, recent=recent, max_len=256)
        target = decode.ToyTarget(cfg, B=3, seed=11)
        gen = np.random.default_rng(3)
        prompts = [gen.integers(0, cfg.vocab, n).tolist() for n in (2, 40, 100)]
        return decode.generate(target, prompts, steps=6, gamma=5)

    whole, _ = run(None)
    assert run(256)[0] == whole
    short, rows = run(32)
    assert all(6 <= len(t) <= 36 for t in short) and max(rows) > 3


def test_a_cache_that_keeps_everything_costs_nothing(decode):
    """Without ``keep`` a step hands the lengths it has to the target, and makes no others."""
    target = decode.ToyTarget(decode.ToyConfig(max_len=256), B=2, seed=12)
    forward, seen = target.forward, []

    def noted(ids, **kw):
        seen.append(kw["prefix_lens"])
        return forward(ids, **kw)

    target.forward = noted
    decode.generate(target, [[1, 2, 3], [4, 5]], steps=3, gamma=4)
    assert len(seen) == 4 and seen[1] is seen[2] is seen[3]


# As in test_gpu_decode: some 8 roundings a layer and 4 outside, of at most half a unit
# relative to the row's largest values, grown by at most 4.
UNIT = {torch.bfloat16: wo.BF16, torch.float32: 2.0 ** -11}  # (fp32 products may run as TF32)


def watched(decode, cfg, B, seed):
    """The model of the decode loop, that compares what the loop hands it with counts of its
    own, its logits with 64 bits over the entries that the caches hold, and the ledger with
    the entries that went in."""
    class Watched(decode.ToyTarget):
        def __init__(self):
            super().__init__(cfg, B, seed=seed)
            self.held, self.now, self.cuts, self.entry = [0] * B, [0] * B, [0] * B, {}

        def forward(self, ids, *, req, pos, cu_seqlens, prefix_lens, totals, status, cache_pos=None):
            cu = cu_seqlens.tolist()
            before = [[entries(c, r, self.held[r]) for r in range(B)] for c in self.caches]
            logits = super().forward(ids, req=req, pos=pos, cu_seqlens=cu_seqlens, prefix_lens=prefix_lens,
                                     totals=totals, status=status, cache_pos=cache_pos)
            assert prefix_lens.tolist() == self.held and int(totals[0]) == cu[-1]
            for r in range(B):
                a, b = cu[r], cu[r + 1]
                n = b - a
                assert req[a:b].tolist() == [r] * n
                assert pos[a:b].tolist() == list(range(self.now[r], self.now[r] + n))
                assert cache_pos[a:b].tolist() == list(range(self.held[r], self.held[r] + n))
                if not n:
                    continue
                want = self.logits64(ids[a:b], self.now[r], [layer[r] for layer in before])
                error = 4 * (8 * cfg.layers + 4) * UNIT[cfg.dtype] / 2 * want.abs().amax(-1, keepdim=True)
                assert bool(((logits[a:b].double() - want).abs() <= error).all()), r
                for i, c in enumerate(self.caches):
                    ks, vs = entries(c, r, self.held[r] + n)
                    for j in range(n):
                        self.entry[i, r, self.now[r] + j] = ks[self.held[r] + j], vs[self.held[r] + j]
            self.rows = [b - a for a, b in zip(cu, cu[1:])]
            return logits

        def logits64(self, ids, now, before):
            c, n, f = self.cfg, ids.numel(), lambda t: t.double()
            x, half = f(self.embed)[ids.long()], c.head_dim // 2
            cos, sin = (t[:, None] for t in f(self.cos_sin[now:now + n]).split(half, 1))
            chain = torch.ones(n, n, device="cuda", dtype=torch.bool).tril()

            def turned(h, w):
                h = h / (h.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * f(w)
                a, b = h[..., :half], h[..., half:]
                return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

            for (old_k, old_v), w_qkv, w_out, (wq, wk) in zip(before, self.w_qkv, self.w_out, self.norms):
                q, k, v = (x @ f(w_qkv)).view(n, -1, c.head_dim).split([c.n_q_heads, c.n_kv_heads, c.n_kv_heads], 1)
                group = c.n_q_heads // c.n_kv_heads
                k, v = (torch.cat(t).repeat_interleave(group, 1) for t in ((old_k, turned(k, wk)), (old_v, v)))
                s = torch.einsum("ihd,jhd->hij", turned(q, wq), k) * c.head_dim ** -0.5
                sees = torch.cat([torch.ones(n, old_k.size(0), device="cuda", dtype=torch.bool), chain], 1)
                o = torch.einsum("hij,jhd->ihd", s.masked_fill(~sees, -math.inf).softmax(-1), v)
                x = x + o.reshape(n, -1) @ f(w_out)
            return x @ f(self.head)

        def accepted(self, counts, *, lens, now, status):
            counts_of = self.rows if counts is None else counts.tolist()
            super().accepted(counts, lens=lens, now=now, status=status)
            for r, n in enumerate(counts_of):
                self.now[r] += n
                self.cuts[r] += self.held[r] + n > cfg.keep
                self.held[r] = min(self.held[r] + n, cfg.keep)
            assert lens.tolist() == self.held and now.tolist() == self.now
            for i, c in enumerate(self.caches):
                for r, (m, t) in enumerate(zip(self.held, self.now)):
                    ks, vs = entries(c, r, m)
                    for h in range(cfg.n_kv_heads):
                        at = c.positions[r, h, :m].tolist()
                        assert len(set(at)) == m and set(range(max(t - cfg.recent, 0), t)) <= set(at)
                        assert all(0 <= p < t for p in at)
                        assert bool((c.weights[r, h, :m] >= 0).all()) and bool((c.weights[r, h, m:] == 0).all())
                        kept = [self.entry[i, r, p] for p in at]
                        if kept:
                            assert torch.equal(ks[:, h], torch.stack([k[h] for k, _ in kept]))
                            assert torch.equal(vs[:, h], torch.stack([v[h] for _, v in kept]))

    return Watched()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_loop_over_caches_that_are_cut(decode, dtype, monkeypatch):
    """Prompts and steps that evict: places, lengths and ledger are those of the tokens so far,
    and every window's logits are the model's over the entries that are left."""
    cfg = decode.ToyConfig(dtype=decode.CACHE_DTYPES[dtype], cache=decode.CACHE_DTYPES[dtype], keep=32, recent=16,
                           max_len=256)
    target = watched(decode, cfg, B=3, seed=11)
    gen = np.random.default_rng(3)
    prompts = [gen.integers(0, cfg.vocab, n).tolist() for n in (2, 40, 100)]
    prompt_cuts, prefill = [], decode.prefill

    def counted(*args):
        cached = prefill(*args)
        prompt_cuts.extend(target.cuts)
        return cached

    monkeypatch.setattr(decode, "prefill", counted)
    tokens, _ = decode.generate(target, prompts, steps=8, gamma=5)
    assert target.now == [len(p) - 1 + len(t) for p, t in zip(prompts, tokens)]
    assert prompt_cuts[2] >= 2 and min(c - p for c, p in zip(target.cuts[1:], prompt_cuts[1:])) >= 2
