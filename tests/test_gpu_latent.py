"""The latent cache: rows written (dspark_latent_append) and attention of drafted tokens
over it (dspark_latent_attention), against their 64-bit definitions."""

import math

import pytest
import torch

import latent_oracle as lo
import window_oracle as wo
from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    require_gpu()
    from confidence_scheduled_speculative_gb300 import api
    return api


I32 = dict(dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ append

APPEND = [
    # rows, heads, latent, rope, page, rows' and cache's type, interleaved, weight
    (1, 1, 512, 64, 16, "bf16", "bf16", True, True),
    (37, 128, 512, 64, 64, "bf16", "bf16", False, True),
    (5, 20, 512, 64, 16, "f32", "f32", True, True),
    (9, 3, 256, 32, 7, "bf16", "f32", False, True),
    (9, 33, 8, 16, 16, "f32", "bf16", True, False),
    (4, 5, 504, 128, 16, "bf16", "bf16", False, True),
    # odd sizes: an element at a time
    (6, 3, 34, 6, 5, "bf16", "bf16", True, True),
    (6, 3, 510, 22, 16, "f32", "f32", False, True),
    (3, 0, 512, 64, 64, "bf16", "bf16", True, True),
    (700, 2, 512, 48, 32, "bf16", "bf16", True, True),
]


@pytest.mark.parametrize("case", APPEND)
def test_append(api, case):
    rows, heads, latent, rope, page, dtype, kind, inter, weighted = case
    gen = torch.Generator().manual_seed(rows)
    g = torch.Generator("cuda").manual_seed(rows)
    dt = wo.DTYPES[dtype]
    pad = 3
    lens = [rows // 3 + 1, rows - rows // 3 + 2]
    c = lo.Latent(gen, kind, [n + 40 for n in lens], page, latent, rope, filled=False, wide=8)
    rnd = lambda *s: (torch.randn(s, generator=g, device="cuda") * 1.5).to(dt)
    x = rnd(rows + pad, latent + rope + 8)[:, :latent + rope]
    req = torch.tensor([int(i >= rows // 3) for i in range(rows)] + [-1] * pad, **I32)
    pos = torch.tensor([40 + i for i in range(rows + pad)], **I32)
    # stored in another order than rotated
    at = torch.tensor([39 + (i if i < rows // 3 else i - rows // 3) for i in range(rows)] + [0] * pad, **I32)
    angle = torch.rand((rows + 50, rope // 2), generator=g, device="cuda") * 6.28
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1)
    w = rnd(latent) if weighted else None
    q = rnd(rows + pad, max(heads, 1), 40 + rope)
    out = torch.full((rows + pad, max(heads, 1), rope + 24), 7.0, device="cuda", dtype=dt)
    status = torch.zeros(1, **I32)
    kw = dict(q_rope=q[..., 40:], q_rope_out=out[..., 24:]) if heads else {}
    api.dspark_latent_append(x, c.lc(), req=req, pos=pos, cache_pos=at, cos_sin=cos_sin, weight=w,
                             interleaved=inter, status=status, **kw)
    torch.cuda.synchronize()
    assert int(status) == 0
    want, tol = wo.norm_rope(x[:rows, None, :latent], w, 1e-6, None, pos[:rows], inter)
    key, key_tol = wo.norm_rope(x[:rows, None, latent:], None, 0, cos_sin, pos[:rows], inter)
    want, tol = torch.cat([want, key], 2)[:, 0], torch.cat([tol, key_tol], 2)[:, 0]
    got = torch.zeros_like(want)
    for r in range(2):
        mine = (req[:rows] == r).nonzero()[:, 0]
        p = at[mine].long()
        got[mine] = c.pages[c.table[r][p // page].long(), p % page].double()
    unit = wo.out_unit(wo.DTYPES[kind])
    assert bool(((got - want).abs() <= tol * (1 + unit) + unit * want.abs()).all())
    # nothing else was touched
    slots = int((c.pool.view(c.pool.size(0) * page, -1) != 0).any(1).sum())
    assert slots == rows and bool((c.pool[..., latent + rope:] == 0).all())
    if heads:
        want, tol = wo.norm_rope(q[:rows, :, 40:], None, 0, cos_sin, pos[:rows], inter)
        unit = wo.out_unit(dt)
        got = out[:rows, :, 24:].double()
        assert bool(((got - want).abs() <= tol * (1 + unit) + unit * want.abs()).all())
        assert bool((out[rows:] == 7).all()) and bool((out[..., :24] == 7).all())


def test_append_in_place_and_totals(api):
    """Queries rotated where they are; rows from totals[0] on are left alone."""
    gen = torch.Generator().manual_seed(1)
    c = lo.Latent(gen, "bf16", [64], 16, filled=False)
    q = torch.randn((6, 4, 192), device="cuda").bfloat16()
    x = torch.randn((6, 576), device="cuda").bfloat16()
    cos_sin = torch.rand((64, 64), device="cuda")
    pos = torch.arange(6, **I32)
    before = q.clone()
    out = torch.zeros((6, 4, 64), device="cuda", dtype=torch.bfloat16)
    status = torch.zeros(1, **I32)
    kw = dict(req=torch.zeros(6, **I32), pos=pos, cos_sin=cos_sin, status=status, totals=torch.tensor([4, 6], **I32))
    api.dspark_latent_append(x, c.lc(), q_rope=q[..., 128:], q_rope_out=out, **kw)
    assert torch.equal(q, before)
    api.dspark_latent_append(x, c.lc(), q_rope=q[..., 128:], **kw)
    assert torch.equal(q[:4, :, 128:], out[:4]) and torch.equal(q[..., :128], before[..., :128])
    assert torch.equal(q[4:], before[4:]) and bool((out[4:] == 0).all())
    assert int((c.pool != 0).any(2).sum()) == 4 and int(status) == 0


def test_append_bad_rows(api):
    """Rows without a place, a request or a rotation: flagged, nothing of theirs stored;
    without a rotation their queries are left alone too."""
    for heads_dim, kind in ((64, "bf16"), (6, "f32")):
        gen = torch.Generator().manual_seed(2)
        c = lo.Latent(gen, kind, [32, 32], 16, 512 if heads_dim == 64 else 10, heads_dim, filled=False)
        c.table[1, 1] = c.n_pages  # no such page
        n = 7
        dim = c.latent + heads_dim
        x = torch.ones((n, dim), device="cuda", dtype=wo.DTYPES[kind])
        q = torch.ones((n, 2, heads_dim), device="cuda", dtype=wo.DTYPES[kind])
        out = torch.full_like(q, 7.0)
        req = torch.tensor([0, 1, 2, 0, 0, 0, 1], **I32)
        pos = torch.tensor([0, 1, 2, 9, -1, 3, 4], **I32)
        at = torch.tensor([0, 20, 1, 2, 3, 32, 3], **I32)
        status = torch.zeros(1, **I32)
        api.dspark_latent_append(x, c.lc(), q_rope=q, q_rope_out=out, req=req, pos=pos, cache_pos=at,
                                 cos_sin=torch.ones((9, heads_dim), device="cuda"), status=status)
        assert int(status) == api.STATUS_BAD_INDEX
        stored = (c.pool != 0).any(2)
        assert int(stored.sum()) == 2 and bool(stored[int(c.table[0, 0]), 0]) and bool(stored[int(c.table[1, 0]), 3])
        left = (out == 7).all(2).all(1)
        assert left.tolist() == [False, False, False, True, True, False, False]


# --------------------------------------------------------------- attention

class Problem:
    def __init__(self, seed, prefix, win, hq, page, kind="bf16", dtype="bf16", latent=512, rope=64, tree=None,
                 pad=3, q_scale=2.0, wide=0, beside=0, **cache):
        gen = torch.Generator().manual_seed(seed)
        g = torch.Generator("cuda").manual_seed(seed)
        self.prefix, self.win, self.hq, self.dtype = prefix, win, hq, wo.DTYPES[dtype]
        self.cache = lo.Latent(gen, kind, [p + w for p, w in zip(prefix, win)], page, latent, rope, wide=wide, **cache)
        self.rows, D = sum(win), latent + rope
        q = torch.randn((self.rows + pad, hq + beside, D), generator=g, device="cuda") * q_scale
        self.q = q.to(self.dtype)[:, :hq]
        self.scale = D ** -0.5
        self.bits = [wo.chain_bits(w) if tree is None else wo.tree_bits(gen, w, tree == "orphans")
                     if w else [] for w in win]
        self.tree = None
        if tree is not None:
            self.tree = torch.cat([wo.as_int32([b for w in self.bits for b in w]),
                                   torch.full((pad,), -1, dtype=torch.int32)]).cuda()
        self.cu = torch.tensor([0] + win, device="cuda").cumsum(0).int()
        self.prefix_lens = torch.tensor(prefix, **I32)
        self.out = torch.full((self.rows + pad, hq + beside, latent), 7.0, device="cuda", dtype=self.dtype)[:, :hq]
        self.lse = torch.full((self.rows + pad, hq), 7.0, device="cuda")
        self.status = torch.zeros(1, **I32)
        # bfloat16 weights where bfloat16 rows run on the tensor cores
        fast = dtype == kind == "bf16" and latent == 512 and rope == 64 and page % 16 == 0
        self.unit = wo.BF16 if fast else 0.0

    def call(self, api, ws=None, lse=True):
        ws = ws if ws is not None else api.workspace(api.dspark_latent_attention_workspace_bytes(self.hq, self.cache.latent))
        api.dspark_latent_attention(self.q, self.cache.lc(), cu_seqlens=self.cu, prefix_lens=self.prefix_lens,
                                    scale=self.scale, out=self.out, lse=self.lse if lse else None,
                                    ancestors=self.tree, workspace=ws, status=self.status)

    def run(self, api, **kw):
        self.call(api, **kw)
        torch.cuda.synchronize()
        return self

    def check(self, skip=()):
        at = 0
        for r, (P, L) in enumerate(zip(self.prefix, self.win)):
            if L and r not in skip:
                want = wo.attention(self.q[at:at + L], self.cache, r, P, L, self.bits[r], self.scale)
                lo.compare(self.out[at:at + L], self.lse[at:at + L], want, self.unit, self.dtype, r)
            at += L
        assert bool((self.out[self.rows:] == 7).all()) and bool((self.lse[self.rows:] == 7).all())
        return self


SHAPES = [
    dict(prefix=[0], win=[1], hq=1, page=16),
    dict(prefix=[0, 5, 0], win=[1, 1, 3], hq=8, page=16),
    # lengths around the tile and page ends; windows of zero
    dict(prefix=[63, 64, 65, 127, 128, 1, 0], win=[1, 1, 1, 1, 17, 0, 0], hq=16, page=64),
    dict(prefix=[15, 16, 17, 31, 48, 200], win=[1, 2, 1, 9, 32, 5], hq=20, page=16),
    # more rows than a tile, tiles that end inside a token, all heads of one token in two
    dict(prefix=[300, 7], win=[32, 20], hq=128, page=32),
    dict(prefix=[129, 1000], win=[31, 3], hq=7, page=128),
    dict(prefix=[511, 90], win=[3, 5], hq=33, page=48),
    dict(prefix=[100, 3], win=[1, 2], hq=200, page=16),
    dict(prefix=[1000, 333], win=[4, 1], hq=65, page=80, wide=8, beside=1),
    # many requests, many splits
    dict(prefix=[(37 * i) % 500 for i in range(70)], win=[i % 6 for i in range(70)], hq=16, page=64),
    dict(prefix=[(91 * i) % 700 for i in range(300)], win=[1 + i % 2 for i in range(300)], hq=8, page=64),
    dict(prefix=[20000, 3], win=[17, 32], hq=16, page=64),
    dict(prefix=[30001], win=[1], hq=64, page=16),
    dict(prefix=[9001, 9001], win=[1, 2], hq=128, page=64),
    # in 32 bits throughout
    dict(prefix=[100, 0], win=[3, 2], hq=4, page=24, kind="f32", dtype="f32"),
    dict(prefix=[100, 9], win=[3, 2], hq=4, page=7, dtype="f32", latent=256, rope=32),
    dict(prefix=[65], win=[5], hq=2, page=1, kind="f32", latent=34, rope=6),
    dict(prefix=[50], win=[4], hq=2, page=16, latent=510, rope=128),
    dict(prefix=[50, 77], win=[4, 1], hq=3, page=20),
    dict(prefix=[50, 77], win=[4, 1], hq=3, page=16, wide=3),
]


@pytest.mark.parametrize("i", range(len(SHAPES)))
@pytest.mark.parametrize("tree", [None, "tree", "orphans"])
def test_attention(api, i, tree):
    p = Problem(100 + i, tree=tree, **SHAPES[i])
    if SHAPES[i].get("wide") == 3:  # strides that are not pieces of 16 bytes
        p.unit = 0.0
    p.run(api).check()
    assert int(p.status) == 0


FAST = dict(hq=16, page=16)
SLOW = dict(hq=3, page=10, kind="f32", dtype="f32", latent=64, rope=16)


@pytest.mark.parametrize("shape", [FAST, SLOW, dict(hq=128, page=64)])
def test_unseen_entries_have_no_effect(api, shape):
    """NaN and infinities behind a request's end, in the rest of its last page and in window
    tokens that a row does not see; rows that do see them get what the formula gives."""
    for value in (math.nan, math.inf, -math.inf):
        p = Problem(200, [70, 33, 0], [5, 9, 4], tree="orphans", **shape)
        used = torch.zeros(p.cache.pages.shape[:2], dtype=torch.bool, device="cuda")
        for r, n in enumerate((75, 42, 4)):
            at = torch.arange(n, device="cuda")
            used[p.cache.table[r][at // p.cache.page].long(), at % p.cache.page] = True
        p.cache.pages[~used] = value
        p.run(api).check()
        assert int(p.status) == 0
        # a token of the window, whole and in its rotated part only
        p.cache.put(0, 72, value)
        p.cache.put(1, 35, value, slice(p.cache.latent, None))
        p.run(api)
        at = 0
        for r, (P, L) in enumerate(zip(p.prefix, p.win)):
            bad = {0: 2, 1: 2}.get(r)
            blind = [i for i in range(L) if bad is None or not p.bits[r][i] >> bad & 1]
            want = wo.attention(p.q[at:at + L], p.cache, r, P, L, p.bits[r], p.scale)
            rows = torch.tensor(blind, device="cuda")
            lo.compare(p.out[at:at + L][rows], p.lse[at:at + L][rows], [t[rows] for t in want], p.unit, p.dtype, r)
            sees = torch.tensor([i for i in range(L) if i not in blind], device="cuda", dtype=torch.long)
            if bad is not None and len(sees):
                got = p.out[at:at + L][sees].double()
                assert torch.equal(torch.isnan(got), torch.isnan(want[0][sees])), (value, r)
            at += L


@pytest.mark.parametrize("shape", [FAST, SLOW])
def test_scores_far_apart(api, shape):
    """Scores of hundreds (one weight is all), of minus infinity's neighbourhood, a scale of
    zero and a negative one."""
    for scale in (40.0, 0.0, -1.0, 1e-30):
        p = Problem(210, [130, 3], [4, 2], **shape)
        p.scale = scale if scale <= 0 or scale < 1e-20 else p.scale * scale
        p.run(api).check()


@pytest.mark.parametrize("shape", [FAST, SLOW])
def test_bad_requests_do_not_disturb_others(api, shape):
    p = Problem(220, [40, 100, 70, 10], [4, 3, 2, 5], **shape)
    p.prefix_lens[1] = 10 ** 6  # past its table
    p.prefix_lens[2] = -1
    p.run(api).check(skip=(1, 2))
    assert int(p.status) == api.STATUS_BAD_INDEX
    p = Problem(221, [40, 100, 70, 10], [4, 3, 2, 5], **shape)
    p.cache.table[1, 2] = p.cache.n_pages + 5
    p.run(api).check(skip=(1,))
    assert int(p.status) == api.STATUS_BAD_INDEX
    p = Problem(222, [40, 100, 10], [4, 33, 5], **shape)  # a window of 33
    p.bits[1] = wo.chain_bits(33)
    p.run(api).check(skip=(1,))
    assert int(p.status) == api.STATUS_BAD_LEN


@pytest.mark.parametrize("longest", [60, 3000])
def test_more_requests_than_threads(api, longest):
    """Whole jobs and split ones, empty and unusable windows among them."""
    n = 900
    win = [(5 * i) % 4 for i in range(n)]
    p = Problem(220, [(53 * i) % 60 for i in range(n - 1)] + [longest], win[:-1] + [2], hq=16, page=64)
    skip = (3, 500)
    for r in skip:
        p.prefix_lens[r] = 1 << 20
    p.run(api).check(skip=skip)
    assert int(p.status) == api.STATUS_BAD_INDEX


def test_two_at_once(api):
    """Calls on two streams, each with its workspace."""
    two = [Problem(222 + i, *shape, hq=64, page=64).run(api).check()
           for i, shape in enumerate([([7000, 300, 12], [1, 9, 4]), ([90, 5000], [17, 2])])]
    first = [(p.out.clone(), p.lse.clone()) for p in two]
    streams = [torch.cuda.Stream() for _ in two]
    spaces = [api.workspace(api.dspark_latent_attention_workspace_bytes(64, 512)) for _ in two]
    for p in two:
        p.out.fill_(7), p.lse.fill_(7)
    torch.cuda.synchronize()
    for _ in range(5):
        for p, s, ws in zip(two, streams, spaces):
            with torch.cuda.stream(s):
                p.call(api, ws)
    torch.cuda.synchronize()
    for p, (out, lse) in zip(two, first):
        assert torch.equal(p.out, out) and torch.equal(p.lse, lse) and int(p.status) == 0


def test_repeated_captured_and_shared_workspace(api):
    """The same bits again, on another stream, in a graph beside a second captured call
    with the same workspace, and without lse."""
    p = Problem(230, [5000, 77, 900], [2, 9, 1], hq=64, page=64).run(api).check()
    first, first_lse = p.out.clone(), p.lse.clone()
    ws = api.workspace(api.dspark_latent_attention_workspace_bytes(64, 512))
    ws.fill_(255)
    side = torch.cuda.Stream()
    p.out.fill_(7)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        p.call(api, ws, lse=False)
    side.synchronize()
    assert torch.equal(p.out, first)
    other = Problem(231, [300, 4000], [3, 1], hq=16, page=16).run(api).check()
    other_out = other.out.clone()
    graphs = []
    for x in (p, other):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.call(api, ws)
        graphs.append(g)
    for _ in range(2):
        p.out.fill_(7), p.lse.fill_(7), other.out.fill_(7)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(p.out, first) and torch.equal(p.lse, first_lse) and torch.equal(other.out, other_out)


def test_refusals(api):
    p = Problem(240, [5], [2], hq=2, page=16)
    ws = api.workspace(api.dspark_latent_attention_workspace_bytes(2, 512))
    kw = dict(cu_seqlens=p.cu, prefix_lens=p.prefix_lens, scale=1.0, workspace=ws, status=p.status)
    with pytest.raises(ValueError, match="q"):
        api.dspark_latent_attention(p.q[..., :500], p.cache.lc(), out=p.out, **kw)
    with pytest.raises(ValueError, match="out"):
        api.dspark_latent_attention(p.q, p.cache.lc(), out=p.q, **kw)
    both = torch.zeros((5, 4, 576), device="cuda", dtype=torch.bfloat16)
    over = both.view(5, -1)[:, :1024].unflatten(1, (2, 512))
    with pytest.raises(api.DsparkError):
        api.dspark_latent_attention(both[:, :2], p.cache.lc(), out=over, **kw)
    beside = both.view(5, -1)[:, 1152:2176].unflatten(1, (2, 512))
    both[:, :2] = p.q
    api.dspark_latent_attention(both[:, :2], p.cache.lc(), out=beside, **kw)
    with pytest.raises(api.DsparkError):
        api.dspark_latent_attention(p.q, p.cache.lc(), out=p.out, **{**kw, "workspace": ws[:64]})
    with pytest.raises(ValueError, match="pages"):
        api.LatentCache(p.cache.pages.half(), p.cache.table, 512)
    with pytest.raises(ValueError, match="latent_dim"):
        api.LatentCache(p.cache.pages, p.cache.table, 576)
    with pytest.raises(ValueError, match="cos_sin"):
        api.dspark_latent_append(p.q[:, 0], p.cache.lc(), req=p.cu, pos=p.cu, cos_sin=torch.zeros((3, 32), device="cuda"),
                                 status=p.status, max_rows=1)
    with pytest.raises(ValueError, match="q_rope_out"):
        api.dspark_latent_append(p.q[:, 0], p.cache.lc(), req=p.cu, pos=p.cu, cos_sin=torch.zeros((3, 64), device="cuda"),
                                 q_rope_out=p.q[..., :64], status=p.status, max_rows=1)


def test_no_rows(api):
    p = Problem(250, [5, 3], [0, 0], hq=2, page=16, pad=0)
    p.run(api)
    none = torch.zeros(0, **I32)
    before = p.cache.pool.clone()
    api.dspark_latent_append(p.q[:, 0], p.cache.lc(), req=none, pos=none, cos_sin=torch.zeros((3, 64), device="cuda"),
                             q_rope=p.q[..., 512:], status=p.status)
    torch.cuda.synchronize()
    assert int(p.status) == 0 and torch.equal(before, p.cache.pool)


@pytest.mark.parametrize("shape", [FAST, SLOW, dict(hq=128, page=64)])
@pytest.mark.parametrize("prefix", [[70, 33], [2500, 1200]])
def test_seen_infinite_elements(api, shape, prefix):
    """One infinite element of an entry makes a score of infinity, of either sign as the query's
    is: 0 times infinity, or NaN throughout, in the prefix as in the window, whole and split."""
    tokens = dict(prefix=prefix, win=[5, 9])
    for value in (math.inf, -math.inf):
        for at in ((prefix[0] - 9, prefix[1] - 1), (prefix[0] + 2, prefix[1] + 4)):
            p = Problem(205, **tokens, **shape)
            for r, (pos, element) in enumerate(zip(at, (3, p.cache.latent - 1))):
                p.cache.put(r, pos, value, element)
            p.run(api).check()
            assert bool(p.out.isnan().any()) and int(p.status) == 0


def test_append_query_outputs_beside_the_queries(api):
    """Parts of the same heads, or of the same rows, that share no element with the queries."""
    gen = torch.Generator().manual_seed(3)
    c = lo.Latent(gen, "bf16", [64], 16, filled=False)
    x = torch.randn((6, 576), device="cuda").bfloat16()
    wide = torch.randn((6, 4, 192), device="cuda").bfloat16()
    status, pos = torch.zeros(1, **I32), torch.arange(6, **I32)
    kw = dict(req=torch.zeros(6, **I32), pos=pos, cos_sin=torch.rand((64, 64), device="cuda"), status=status)
    want = torch.zeros((6, 4, 64), device="cuda", dtype=torch.bfloat16)
    api.dspark_latent_append(x, c.lc(), q_rope=wide[..., 128:], q_rope_out=want, **kw)
    before = wide.clone()
    api.dspark_latent_append(x, c.lc(), q_rope=wide[..., 128:], q_rope_out=wide[..., 64:128], **kw)
    assert torch.equal(wide[..., 64:128], want) and torch.equal(wide[..., 128:], before[..., 128:])
    assert torch.equal(wide[..., :64], before[..., :64])
    rows = torch.cat([before.flatten(1), torch.zeros((6, 256), device="cuda", dtype=torch.bfloat16)], 1)
    out = rows[:, 768:].unflatten(1, (4, 64))
    api.dspark_latent_append(x, c.lc(), q_rope=rows[:, :768].unflatten(1, (4, 192))[..., 128:], q_rope_out=out, **kw)
    assert torch.equal(out, want) and torch.equal(rows[:, :768], before.flatten(1)) and int(status) == 0
    with pytest.raises(api.DsparkError):
        api.dspark_latent_append(x, c.lc(), q_rope=wide[..., 128:], q_rope_out=wide[..., 120:184], **kw)
    assert torch.equal(wide[..., 128:], before[..., 128:])


@pytest.mark.parametrize("shape", [FAST, dict(hq=128, page=64)])
def test_unseen_entries_have_no_effect_on_split_jobs(api, shape):
    """As test_unseen_entries_have_no_effect, where a job's parts are joined: NaN and infinities
    of the window reach the rows that see them, through the join, and no others."""
    for value in (math.nan, math.inf, -math.inf):
        p = Problem(206, [2500, 1200, 0], [5, 9, 4], tree="orphans", **shape)
        used = torch.zeros(p.cache.pages.shape[:2], dtype=torch.bool, device="cuda")
        for r, n in enumerate((2505, 1209, 4)):
            at = torch.arange(n, device="cuda")
            used[p.cache.table[r][at // p.cache.page].long(), at % p.cache.page] = True
        p.cache.pages[~used] = value
        p.run(api).check()
        p.cache.put(0, 2502, value, 5)
        p.cache.put(1, 1202, value, 300)
        p.run(api).check()
        assert bool(p.out.isnan().any()) and bool(p.out.isfinite().any()) and int(p.status) == 0


def team(p, pairs):
    """How many pairs of CTAs go through the positions together: the largest of 1, 2 and 4 whose
    members' steps are an eighth more at most than those of pairs alone."""
    def steps(size):
        return sum((-(-(P + L) // 128) + 2) * -(-(-(-L * p.hq // 128)) // size)
                   for P, L in zip(p.prefix, p.win) if L)
    return max(s for s in (1, 2, 4) if s == 1 or steps(s) * 8 * pairs <= steps(1) * 9 * (pairs // s))


@pytest.mark.parametrize("size,prefix,win,hq", [
    (4, [2500], [32], 64),
    # 15, 16 and 1 row tiles: groups that leave one member idle, or three
    (4, [2500, 700], [30, 32], 64),
    (4, [6000, 90, 3000], [32, 1, 31], 64),
    (2, [2500], [2], 128),
    # 9, 2 and 9 row tiles, and 13
    (2, [3000, 40, 900], [9, 2, 9], 128),
    (2, [7000, 600], [13, 3], 128),
])
@pytest.mark.parametrize("tree", [None, "orphans"])
def test_teams(api, size, prefix, win, hq, tree):
    """Pairs of CTAs that go through the same positions in teams, members without a row tile,
    and the join of their parts."""
    p = Problem(260 + size, prefix, win, hq=hq, page=64, tree=tree)
    assert {team(p, pairs) for pairs in range(72, 77)} == {size}
    ws = api.workspace(api.dspark_latent_attention_workspace_bytes(hq, 512))
    ws.fill_(255)
    p.run(api, ws=ws).check()
    first, first_lse = p.out.clone(), p.lse.clone()
    p.out.fill_(7), p.lse.fill_(7)
    p.run(api, ws=ws)
    assert torch.equal(p.out, first) and torch.equal(p.lse, first_lse) and int(p.status) == 0
