"""A cache that is kept short: gathered attention weights (dspark_attention_weights) and
eviction (dspark_kv_evict), against their definitions."""

import math

import pytest
import torch

import latent_oracle as lo
import window_oracle as wo
from gpu_helpers import require_gpu
from test_gpu_attention import Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    require_gpu()
    from confidence_scheduled_speculative_gb300 import api
    return api


I32 = dict(dtype=torch.int32, device="cuda")


# --------------------------------------------------------------- gathering

class Gathering(Problem):
    """The attention's problem, attended to, with a ledger beside it."""

    def __init__(self, api, seed, counts=None, more=5, decay=0.75, **kw):
        super().__init__(seed, **kw)
        self.run(api)
        B, hkv = len(self.win), self.cache.heads
        self.counts = self.win if counts is None else counts
        self.n_counts = None if counts is None else torch.tensor(counts, **I32)
        S = self.length = max(p + c for p, c in zip(self.prefix, self.counts)) + more
        g = torch.Generator("cuda").manual_seed(seed)
        self.before = torch.rand((B, hkv, S), generator=g, device="cuda")
        self.weights = torch.full_like(self.before, 9.0)
        self.positions = torch.full((B, hkv, S), -5, **I32)
        self.pos = 1000 + torch.arange(self.q.size(0), **I32)
        self.decay = decay

    def gather(self, api, into=None, **kw):
        api.dspark_attention_weights(
            self.q, self.cache.kv(), lse=self.lse, cu_seqlens=self.cu, prefix_lens=self.prefix_lens,
            scale=self.scale, ancestors=self.tree, counts=self.n_counts, decay=self.decay, weights=self.before,
            weights_out=self.weights if into is None else into, pos=self.pos, positions=self.positions,
            status=self.status, **kw)
        torch.cuda.synchronize()
        return self

    def check(self, skip=()):
        at = 0
        for r, (P, L, n) in enumerate(zip(self.prefix, self.win, self.counts)):
            if r not in skip:
                e, tol = lo.gathered(self.q[at:at + L], self.lse[at:at + L], self.cache, r, P, L, n, self.bits[r],
                                     self.scale)
                want = e.clone()
                want[:, :P] += self.decay * self.before[r, :, :P].double()
                got = self.weights[r].double()
                off = (got[:, :P + n] - want).abs() - (tol + 3 * wo.U32 * want.abs() + 1e-38)
                assert not off.numel() or float(off.max()) <= 0, (r, float(off.max()))
                assert bool((got[:, P + n:] == 0).all())
                noted = torch.full_like(self.positions[r], -5)
                noted[:, P:P + n] = self.pos[at:at + n]
                assert torch.equal(self.positions[r], noted), r
            at += L
        return self


SHAPES = [
    dict(prefix=[0], win=[1], hq=1, hkv=1, D=64, page=16, kind="bf16"),
    dict(prefix=[0, 5, 0, 9], win=[1, 1, 3, 0], hq=8, hkv=2, D=64, page=16, kind="bf16"),
    dict(prefix=[63, 64, 65, 127, 128, 1], win=[1, 1, 1, 1, 17, 0], hq=8, hkv=1, D=128, page=64, kind="bf16"),
    dict(prefix=[15, 16, 17, 31, 48, 200], win=[1, 2, 1, 9, 32, 5], hq=12, hkv=4, D=128, page=16, kind="bf16"),
    dict(prefix=[300, 7], win=[32, 20], hq=16, hkv=2, D=128, page=32, kind="e4m3"),
    dict(prefix=[129, 1], win=[31, 1], hq=7, hkv=1, D=64, page=128, kind="e4m3"),
    dict(prefix=[90], win=[32], hq=40, hkv=1, D=128, page=16, kind="bf16"),
    dict(prefix=[1000, 333], win=[4, 1], hq=20, hkv=4, D=128, page=80, kind="e4m3"),
    dict(prefix=[700], win=[13], hq=6, hkv=2, D=64, page=256, kind="bf16", layout="heads"),
    dict(prefix=[(37 * i) % 500 for i in range(70)], win=[i % 6 for i in range(70)], hq=8, hkv=2, D=128, page=64,
         kind="bf16"),
    dict(prefix=[9000, 3], win=[17, 32], hq=8, hkv=1, D=128, page=64, kind="e4m3"),
    dict(prefix=[100, 0], win=[3, 2], hq=4, hkv=2, D=80, page=24, kind="f32", dtype="f32"),
    dict(prefix=[65], win=[5], hq=2, hkv=1, D=34, page=1, kind="e4m3", dtype="f32"),
    dict(prefix=[50], win=[4], hq=2, hkv=1, D=256, page=7, kind="bf16"),
]


@pytest.mark.parametrize("i", range(len(SHAPES)))
@pytest.mark.parametrize("tree", [None, "tree", "orphans"])
def test_gathered(api, i, tree):
    win = SHAPES[i]["win"]
    p = Gathering(api, 400 + i, tree=tree, **SHAPES[i]).gather(api).check()
    assert int(p.status) == 0
    p = Gathering(api, 430 + i, counts=[(3 * k) % (w + 1) for k, w in enumerate(win, 1)], tree=tree, **SHAPES[i])
    first = p.gather(api).check().weights.clone()
    assert int(p.status) == 0
    into = p.before  # in place, and the same bits
    p.gather(api, into=into)
    assert torch.equal(into, first)


def test_gathered_over_what_is_unseen(api):
    """NaN behind the end and in window tokens that the counted rows do not see."""
    for kind in ("bf16", "e4m3"):
        p = Gathering(api, 450, tree="orphans", prefix=[70, 33], win=[5, 9], hq=8, hkv=2, D=128, page=16, kind=kind)
        p.cache.put("k", 0, 74, math.nan)
        p.bits[0] = [b & ~16 for b in p.bits[0]]
        p.tree[:5] &= ~16
        last = int(p.cache.table[1, 2])
        p.cache.k[last, 42 - 32:] = torch.tensor(math.nan, device="cuda").to(p.cache.k.dtype)
        p.run(api)
        p.cache.put("v", 0, 74, 1.0)
        p.gather(api)
        p.cache.put("k", 0, 74, 1.0)  # the definition multiplies
        p.check()


def test_gathered_over_an_infinite_key(api):
    """A key of -inf under queries above zero: s = -inf, which adds nothing."""
    for D, hq in ((128, 5), (64, 8), (80, 3)):
        p = Gathering(api, 470, prefix=[40], win=[1], hq=hq, hkv=1, D=D, page=16, kind="bf16")
        p.q.copy_(p.q.abs() + 0.01)
        p.cache.put("k", 0, 7, -math.inf)
        p.run(api)
        p.gather(api)
        assert float(p.weights[0, 0, 7]) == float(p.before[0, 0, 7] * p.decay)  # (rounded once, both)
        assert bool(p.weights.isfinite().all()) and int(p.status) == 0


def test_gathering_bad_requests(api):
    kw = dict(hq=8, hkv=2, D=128, page=64, kind="bf16")
    p = Gathering(api, 460, prefix=[40, 100, 70], win=[4, 3, 2], counts=[4, 3, 2], **kw)
    p.n_counts[1] = 4
    p.gather(api).check(skip=(1,))
    assert int(p.status) == api.STATUS_BAD_LEN and bool((p.weights[1] == 9).all())
    p = Gathering(api, 461, prefix=[40, 100, 70], win=[4, 3, 2], more=0, **kw)
    p.prefix_lens[1] = 101
    p.gather(api).check(skip=(1,))
    assert int(p.status) == api.STATUS_CAPACITY and bool((p.weights[1] == 9).all())
    p = Gathering(api, 462, prefix=[40, 100, 70], win=[4, 3, 2], **kw)
    p.cache.table[1, 0] = -1
    p.gather(api).check(skip=(1,))
    assert int(p.status) == api.STATUS_BAD_INDEX


# ---------------------------------------------------------------- eviction

class Evicting:
    def __init__(self, seed, lens, keep, recent, hkv=2, D=64, page=16, kind="bf16", layout="tokens", more=3,
                 spread=2.0, ties=False):
        gen = torch.Generator().manual_seed(seed)
        g = torch.Generator("cuda").manual_seed(seed)
        self.lens, self.keep, self.recent = lens, keep, recent
        self.cache = wo.Cache(gen, kind, lens, hkv, D, page, layout)
        B, S = len(lens), max(lens) + more
        self.length, self.hkv = S, hkv
        w = torch.exp(spread * torch.randn((B, hkv, S), generator=g, device="cuda"))
        if ties:
            w = torch.where(w < 1, 0.0, w.clamp(max=3.0).round())
        self.weights = w
        order = torch.rand((B, hkv, S), generator=g, device="cuda")
        self.positions = torch.argsort(order, dim=-1).to(torch.int32) * 2
        self.now = torch.tensor([2 * n for n in lens], **I32)
        self.n = torch.tensor(lens, **I32)
        self.status = torch.zeros(1, **I32)

    def run(self, api, inplace=False):
        ws = api.workspace(api.dspark_kv_evict_workspace_bytes(len(self.lens), self.hkv, self.length))
        ws.fill_(255)
        self.was = [t.clone() for t in (self.cache.k.view(torch.uint8), self.cache.v.view(torch.uint8))]
        self.was_scale = [None if t is None else t.clone() for t in (self.cache.k_scale, self.cache.v_scale)]
        self.w, self.p = self.weights.clone(), self.positions.clone()
        out = dict(weights_out=self.w, positions_out=self.p, new_lens=torch.full_like(self.n, -1))
        kw = dict(lens=self.n, weights=self.weights, positions=self.positions)
        if inplace:
            kw = dict(lens=self.n.clone(), weights=self.w, positions=self.p)
            out = {}
        else:
            self.w.fill_(9), self.p.fill_(9)
        api.dspark_kv_evict(self.cache.kv(), now=self.now, keep=self.keep, recent=self.recent, workspace=ws,
                            status=self.status, **kw, **out)
        torch.cuda.synchronize()
        self.new = kw["lens"] if inplace else out["new_lens"]
        return self

    def check(self, skip=()):
        c = self.cache
        want = [t.clone() for t in self.was]
        want_scale = [None if t is None else t.clone() for t in self.was_scale]
        kept = []
        for r, n in enumerate(self.lens):
            if r in skip:
                continue
            assert int(self.new[r]) == min(n, self.keep)
            for h in range(self.hkv):
                w, p = self.weights[r, h], self.positions[r, h]
                of = lo.evicted(w.tolist(), p.tolist(), n, int(self.now[r]), self.keep, self.recent)
                kept.append(of)
                idx = torch.tensor(of, device="cuda", dtype=torch.long)
                for got, src in ((self.w, w), (self.p, p)):
                    line = torch.zeros_like(src)
                    line[:len(of)] = src[idx]
                    same = (got[r, h] == line) | (torch.isnan(got[r, h].float()) & torch.isnan(line.float()))
                    assert bool(same.all()), (r, h)
                moved = [(i, j) for i, j in enumerate(of) if i != j]
                if not moved:
                    continue
                a, b = (torch.tensor(x, device="cuda") for x in zip(*moved))
                pa, ta, pb, tb = (x.long() for x in (c.table[r][a // c.page], a % c.page, c.table[r][b // c.page],
                                                     b % c.page))
                for t, s in zip(want, self.was):
                    t[pa, ta, h] = s[pb, tb, h]
                for t, s in zip(want_scale, self.was_scale):
                    if t is not None:
                        t[pa, h, ta] = s[pb, h, tb]
        if not skip:
            assert torch.equal(c.k.view(torch.uint8), want[0]) and torch.equal(c.v.view(torch.uint8), want[1])
            if want_scale[0] is not None:
                assert torch.equal(c.k_scale, want_scale[0]) and torch.equal(c.v_scale, want_scale[1])
        return kept


EVICT = [
    dict(lens=[1], keep=1, recent=0, hkv=1),
    dict(lens=[0, 1, 2, 3, 5, 17], keep=2, recent=1),
    dict(lens=[40, 64, 65, 100], keep=64, recent=16),
    dict(lens=[300, 20, 299], keep=200, recent=200),
    dict(lens=[300, 20, 299], keep=20, recent=0, kind="e4m3", D=128, page=64),
    dict(lens=[1023, 1024, 1025, 2500], keep=1000, recent=100, hkv=1, page=128),
    dict(lens=[5000, 33000], keep=4096, recent=1024, hkv=1, page=64, kind="e4m3"),
    # two and eight CTAs a line, and longer than they hold
    dict(lens=[20000, 17, 16385], keep=9000, recent=50, D=64, page=64),
    dict(lens=[100000, 131040], keep=50000, recent=4096, hkv=1, page=128, kind="e4m3"),
    dict(lens=[70001], keep=69990, recent=5, hkv=1, page=64, ties=True),
    dict(lens=[140000, 500], keep=64000, recent=64000, hkv=1, page=64, kind="e4m3"),
    dict(lens=[400000, 393217], keep=200000, recent=100, hkv=1, D=16, page=256, spread=0.1),
    dict(lens=[700, 90], keep=80, recent=8, ties=True),
    dict(lens=[3000], keep=1500, recent=10, ties=True, spread=0.5),
    dict(lens=[300, 120], keep=64, recent=16, layout="heads", hkv=3),
    dict(lens=[90, 33], keep=31, recent=3, D=34, page=7, kind="f32"),
    dict(lens=[90, 33], keep=31, recent=3, D=34, page=7, kind="e4m3"),
    dict(lens=[90, 33], keep=31, recent=3, D=34, page=7, kind="bf16"),
]


@pytest.mark.parametrize("i", range(len(EVICT)))
@pytest.mark.parametrize("inplace", [False, True])
def test_evict(api, i, inplace):
    e = Evicting(500 + i, **EVICT[i]).run(api, inplace)
    e.check()
    assert int(e.status) == 0


def test_gather_and_evict_captured(api):
    """One graph of a gathering and an eviction in place, replayed over lengths that change
    between: the same bits as the calls themselves, with a workspace that two graphs share."""
    def state():
        p = Gathering(api, 470, prefix=[200, 90], win=[5, 3], hq=8, hkv=2, D=128, page=16, kind="e4m3", more=40)
        p.positions = torch.arange(p.length, **I32).repeat(2, 2, 1)
        p.lens = torch.zeros(2, **I32)
        return p

    def calls(p, ws):
        api.dspark_attention_weights(p.q, p.kv, lse=p.lse, cu_seqlens=p.cu, prefix_lens=p.prefix_lens,
                                     scale=p.scale, weights=p.before, pos=p.pos, positions=p.positions,
                                     status=p.status)
        api.dspark_kv_evict(p.kv, lens=p.lens, now=p.now, keep=64, recent=8, weights=p.before,
                            positions=p.positions, workspace=ws, status=p.status)

    def rounds(p, go):
        for n in ([200, 90], [64, 64], [64, 50]):
            p.prefix_lens.copy_(torch.tensor(n, **I32))
            p.lens.copy_(p.prefix_lens + torch.tensor([5, 3], **I32))
            p.now.copy_(p.lens)
            go()
        torch.cuda.synchronize()
        assert int(p.status) == 0
        return [t.clone() for t in (p.before, p.positions, p.lens, p.cache.k.view(torch.uint8),
                                    p.cache.v.view(torch.uint8), p.cache.k_scale, p.cache.v_scale)]

    ws = api.workspace(api.dspark_kv_evict_workspace_bytes(2, 2, state().length))
    results = []
    for captured in (False, True, True):
        p = state()
        p.kv, p.now = p.cache.kv(), torch.zeros(2, **I32)
        if captured:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                calls(p, ws)
            results.append(rounds(p, g.replay))
        else:
            results.append(rounds(p, lambda: calls(p, ws)))
    for got in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got, results[0]))


def test_evict_two_at_once(api):
    """Evictions on two streams, of several CTAs a line and of one, each with its workspace."""
    two = [Evicting(525, [100000, 60000], keep=30000, recent=4096, hkv=2, page=128, kind="e4m3"),
           Evicting(526, [3000, 8000, 100], keep=700, recent=64, hkv=4)]
    streams = [torch.cuda.Stream() for _ in two]
    torch.cuda.synchronize()
    kept = []
    for e, s in zip(two, streams):
        e.was = [t.clone() for t in (e.cache.k.view(torch.uint8), e.cache.v.view(torch.uint8))]
        e.was_scale = [None if t is None else t.clone() for t in (e.cache.k_scale, e.cache.v_scale)]
        e.w, e.p, e.new = e.weights.clone(), e.positions.clone(), e.n.clone()
        kept.append((e, s, e.cache.kv(), api.workspace(
            api.dspark_kv_evict_workspace_bytes(len(e.lens), e.hkv, e.length))))
    torch.cuda.synchronize()
    for e, s, kv, ws in kept:
        with torch.cuda.stream(s):
            api.dspark_kv_evict(kv, lens=e.new, now=e.now, keep=e.keep, recent=e.recent, weights=e.w, positions=e.p,
                                workspace=ws, status=e.status)
    torch.cuda.synchronize()
    for e in two:
        e.check()
        assert int(e.status) == 0


def test_evict_odd_weights(api):
    """NaN, infinities, negative and equal weights, -0 beside 0; every entry fresh, and
    positions at the ends of their range."""
    e = Evicting(520, [64, 64, 64], keep=40, recent=8, hkv=1)
    e.weights[0, 0, ::3] = math.nan
    e.weights[0, 0, 1::6] = math.inf
    e.weights[0, 0, 2::6] = -math.inf
    e.weights[0, 0, 5::12] = -1.5
    e.weights[1] = 0.0
    e.weights[1, 0, ::2] = -0.0
    e.now[1] = -2 ** 31
    e.now[2] = 2 ** 31 - 1
    e.run(api).check()
    assert int(e.status) == api.STATUS_BAD_INPUT


def test_evict_bad_requests(api):
    e = Evicting(530, [64, 80, 50], keep=32, recent=8)
    e.n[1] = e.length + 1
    e.run(api).check(skip=(1,))
    assert int(e.status) == api.STATUS_BAD_LEN
    assert int(e.new[1]) == e.length + 1 and bool((e.w[1] == 9).all())
    e = Evicting(531, [64, 80], keep=32, recent=8)
    e.cache.table[1, 0] = e.cache.n_pages
    e.run(api).check(skip=(1,))
    assert int(e.status) == api.STATUS_BAD_INDEX


def test_evict_refusals(api):
    e = Evicting(540, [40], keep=32, recent=8)
    ws = api.workspace(api.dspark_kv_evict_workspace_bytes(1, 2, e.length))
    kw = dict(lens=e.n, now=e.now, weights=e.weights, positions=e.positions, workspace=ws, status=e.status)
    for bad in (dict(keep=0, recent=0), dict(keep=4, recent=5), dict(keep=4, recent=-1)):
        with pytest.raises(api.DsparkError):
            api.dspark_kv_evict(e.cache.kv(), **kw, **bad)
    with pytest.raises(api.DsparkError):
        api.dspark_kv_evict(e.cache.kv(), keep=4, recent=1, **{**kw, "workspace": ws[:256]})
    with pytest.raises(ValueError, match="positions"):
        api.dspark_kv_evict(e.cache.kv(), keep=4, recent=1, **{**kw, "positions": e.positions[:, :, 1:]})
    with pytest.raises(ValueError, match="weights"):
        api.dspark_kv_evict(e.cache.kv(), keep=4, recent=1, **{**kw, "weights": e.weights[0]})


@pytest.mark.parametrize("case", [
    # one CTA a line of more than 8192 places: a short ledger, and many lines
    dict(lens=[10000, 8200, 9999], keep=4096, recent=64, hkv=1, page=64),
    dict(lens=[9500, 3], keep=9000, recent=9000, hkv=2, page=64, ties=True),
    dict(lens=[500 * i + 700 for i in range(19)] + [40000], keep=3000, recent=100, hkv=4, D=16, page=64, kind="e4m3"),
])
@pytest.mark.parametrize("inplace", [False, True])
def test_evict_one_cta_a_line(api, case, inplace):
    e = Evicting(550, **case).run(api, inplace)
    e.check()
    assert int(e.status) == 0


@pytest.mark.parametrize("case", [
    # spans of 512 and of 2048 positions, and more rows than are multiplied at a time
    dict(prefix=[8990, 700, 33] + [(91 * i) % 400 for i in range(17)], win=[9, 5, 32] + [i % 3 for i in range(17)],
         hq=32, hkv=2, D=128, page=64),
    dict(prefix=[8200, 4095] + [(37 * i) % 300 for i in range(38)], win=[9, 7] + [i % 6 for i in range(38)],
         hq=128, hkv=8, D=64, page=64),
])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_gathered_over_long_spans(api, case, kind):
    p = Gathering(api, 490, tree="tree", kind=kind, **case)
    blocks = -(-(p.length * case["hkv"] * len(p.win) // (8 * 152)) // 256)
    assert blocks >= (8 if case["hkv"] == 8 else 2)
    p.gather(api).check()
    assert int(p.status) == 0
