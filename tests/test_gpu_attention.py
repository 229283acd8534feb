"""Attention of drafted tokens over a paged cache (dspark_tree_attention)
against its 64-bit definition."""

import math

import pytest
import torch

import window_oracle as wo
from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


@pytest.fixture(scope="module")
def api(dev):
    from confidence_scheduled_speculative_gb300 import api
    return api


class Problem:
    def __init__(self, seed, prefix, win, hq, hkv, D, page, kind, dtype="bf16", layout="tokens",
                 tree=None, pad=3, q_scale=2.0, **cache):
        gen = torch.Generator().manual_seed(seed)
        g = torch.Generator("cuda").manual_seed(seed)
        self.prefix, self.win, self.hq, self.D, self.dtype = prefix, win, hq, D, wo.DTYPES[dtype]
        self.cache = wo.Cache(gen, kind, [p + w for p, w in zip(prefix, win)], hkv, D, page, layout,
                              **cache)
        self.rows = sum(win)
        # the queries lie beside other columns, as in a projection's output
        wide = torch.randn((self.rows + pad, hq + 1, D), generator=g, device="cuda") * q_scale
        self.q = wide.to(self.dtype)[:, :hq]
        self.scale = D ** -0.5
        self.bits = [wo.chain_bits(w) if tree is None else wo.tree_bits(gen, w, tree == "orphans")
                     if w else [] for w in win]
        self.tree = None
        if tree is not None:
            self.tree = torch.cat([wo.as_int32([b for w in self.bits for b in w]),
                                   torch.full((pad,), -1, dtype=torch.int32)]).cuda()
        i32 = dict(dtype=torch.int32, device="cuda")
        self.cu = torch.tensor([0] + win, device="cuda").cumsum(0).int()
        self.prefix_lens = torch.tensor(prefix, **i32)
        self.out = torch.full((self.rows + pad, hq, D), 7.0, device="cuda", dtype=self.dtype)
        self.lse = torch.full((self.rows + pad, hq), 7.0, device="cuda")
        self.status = torch.zeros(1, **i32)

    def run(self, api, lse=True):
        ws = api.workspace(api.dspark_tree_attention_workspace_bytes(self.hq, self.D))
        api.dspark_tree_attention(self.q, self.cache.kv(), cu_seqlens=self.cu,
                                  prefix_lens=self.prefix_lens, scale=self.scale, out=self.out,
                                  lse=self.lse if lse else None, ancestors=self.tree, workspace=ws,
                                  status=self.status)
        torch.cuda.synchronize()
        return self

    def unit(self):
        """The rounding of the weights: to the 16-bit type of the products
        (bfloat16, or half for the 8-bit cache) where bfloat16 rows run on the
        tensor cores."""
        if self.dtype != torch.bfloat16 or self.cache.kind == "f32":
            return 0.0
        return wo.BF16 if self.cache.kind == "bf16" else wo.F16

    def smallest_weight(self, r, n):
        """What weights lose as halves where they are far below the largest (of weight
        times scale): half of the smallest step 2^-24, taken 2^6 finer, of codes up
        to 448, for each of n positions."""
        if self.dtype != torch.bfloat16 or self.cache.kind != "e4m3":
            return 0.0
        page, tok = self.cache.slots(r, 0, n)
        return n * 2.0 ** -31 * 448 * float(self.cache.v_scale[page, :, tok].abs().max())

    def check(self, skip=(), far_below=False):
        lo = 0
        for r, (P, L) in enumerate(zip(self.prefix, self.win)):
            if L and r not in skip:
                o, lse, tol, lse_tol, o_abs = wo.attention(self.q[lo:lo + L], self.cache, r, P, L,
                                                           self.bits[r], self.scale)
                got, got_lse = self.out[lo:lo + L].double(), self.lse[lo:lo + L].double()
                assert torch.equal(torch.isnan(got), torch.isnan(o)), r
                assert torch.equal(torch.isinf(got), torch.isinf(o)), r
                fine = torch.isfinite(o)
                u = self.unit()
                bound = (tol + u * o_abs) * (1 + wo.BF16) + wo.out_unit(self.dtype) * o.abs() + 1e-38
                if far_below:
                    bound = bound + self.smallest_weight(r, P + L)
                off = ((got - o).abs() - bound)[fine]
                assert not off.numel() or float(off.max()) <= 0, (r, float(off.max()))
                assert torch.equal(got_lse == -math.inf, lse == -math.inf), r
                fine = torch.isfinite(lse)
                off = ((got_lse - lse).abs() - lse_tol)[fine]
                assert not off.numel() or float(off.max()) <= 0, (r, float(off.max()))
            lo += L
        assert bool((self.out[self.rows:] == 7).all()) and bool((self.lse[self.rows:] == 7).all())


SHAPES = [
    # one token, no prefix; the smallest window of all
    dict(prefix=[0], win=[1], hq=1, hkv=1, D=64, page=16, kind="bf16"),
    dict(prefix=[0, 5, 0], win=[1, 1, 3], hq=8, hkv=2, D=64, page=16, kind="bf16"),
    # lengths around the tile and page ends; windows of zero
    dict(prefix=[63, 64, 65, 127, 128, 1, 0], win=[1, 1, 1, 1, 17, 0, 0], hq=8, hkv=1, D=128,
         page=64, kind="bf16"),
    dict(prefix=[15, 16, 17, 31, 48, 200], win=[1, 2, 1, 9, 32, 5], hq=12, hkv=4, D=128, page=16,
         kind="bf16"),
    # more rows than a tile: 32 tokens of 8, 7, 16 and 40 heads a key head
    dict(prefix=[300, 7], win=[32, 20], hq=16, hkv=2, D=128, page=32, kind="bf16"),
    dict(prefix=[129], win=[31], hq=7, hkv=1, D=64, page=128, kind="bf16"),
    dict(prefix=[511], win=[32], hq=32, hkv=2, D=64, page=48, kind="bf16"),
    dict(prefix=[90], win=[32], hq=40, hkv=1, D=128, page=16, kind="e4m3"),
    # pages that a tile does not divide, larger and smaller ones
    dict(prefix=[1000, 333], win=[4, 1], hq=4, hkv=4, D=128, page=80, kind="bf16"),
    dict(prefix=[1000, 333], win=[4, 1], hq=4, hkv=4, D=64, page=112, kind="e4m3"),
    dict(prefix=[700], win=[13], hq=6, hkv=2, D=128, page=256, kind="e4m3"),
    # many requests, many splits
    dict(prefix=[(37 * i) % 500 for i in range(70)], win=[i % 6 for i in range(70)], hq=4, hkv=2,
         D=128, page=64, kind="bf16"),
    dict(prefix=[(91 * i) % 1500 for i in range(300)], win=[1 + i % 2 for i in range(300)], hq=8,
         hkv=1, D=128, page=64, kind="e4m3"),
    dict(prefix=[20000, 3], win=[17, 32], hq=8, hkv=1, D=128, page=64, kind="bf16"),
    dict(prefix=[30001], win=[1], hq=16, hkv=2, D=128, page=16, kind="e4m3"),
    # 32-bit rows, other head and page sizes: in 32 bits throughout
    dict(prefix=[100, 0], win=[3, 2], hq=4, hkv=2, D=80, page=24, kind="f32", dtype="f32"),
    dict(prefix=[100, 9], win=[3, 2], hq=4, hkv=2, D=256, page=7, kind="bf16", dtype="f32"),
    dict(prefix=[65], win=[5], hq=2, hkv=1, D=34, page=1, kind="e4m3", dtype="f32"),
    dict(prefix=[65, 2], win=[5, 4], hq=2, hkv=1, D=128, page=16, kind="f32", dtype="bf16"),
    dict(prefix=[50], win=[4], hq=2, hkv=1, D=96, page=16, kind="bf16", dtype="bf16"),
    dict(prefix=[50], win=[4], hq=2, hkv=1, D=128, page=20, kind="e4m3", dtype="bf16"),
]


@pytest.mark.parametrize("i", range(len(SHAPES)))
@pytest.mark.parametrize("tree", [None, "tree", "orphans"])
def test_attention(api, dev, i, tree):
    p = Problem(100 + i, tree=tree, **SHAPES[i]).run(api)
    p.check()
    assert int(p.status) == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
def test_heads_before_tokens(api, dev, kind, D):
    p = Problem(3, [77, 130, 64], [5, 1, 32], 8, 2, D, 32, kind, layout="heads").run(api)
    p.check()


@pytest.mark.parametrize("kind,dtype,page", [("bf16", "bf16", 16), ("e4m3", "bf16", 64), ("f32", "f32", 16)])
def test_what_is_not_seen_has_no_effect(api, dev, kind, dtype, page):
    """NaN past a request's end, in pages of no request, in window tokens that
    a row does not see; a request next to one whose prefix holds a NaN."""
    for bad in (math.nan, math.inf):
        p = Problem(8, [37, 64, 5, 90], [6, 9, 12, 3], 8, 2, 128, page, kind, dtype=dtype,
                    tree="orphans", spare=1)
        c = p.cache
        used = torch.zeros((c.n_pages, page), dtype=torch.bool, device="cuda")
        for r, (P, L) in enumerate(zip(p.prefix, p.win)):
            g, t = c.slots(r, 0, P + L)
            used[g, t] = True
        for t in (c.k, c.v):
            if kind == "e4m3":
                t.view(torch.uint8)[~used] = 0x7F
            else:
                t[~used] = bad
        for s in (c.k_scale, c.v_scale):
            if s is not None:
                s.masked_fill_(~used[:, None, :], bad)
        for which in ("k", "v"):
            c.put(which, 1, 64 + 4, bad)     # one window token of request 1
            c.put(which, 3, 20, math.nan)    # request 3's prefix: its rows are NaN
        c.put("v", 2, 5 + 7, -bad)
        p.run(api).check()
        assert int(p.status) == 0


def test_large_scores(api, dev):
    """Scores of thousands, rising and falling along the prefix, so that the
    running maximum moves at every tile or never."""
    for slope in (1, -1):
        for kind in ("bf16", "e4m3"):
            p = Problem(9, [700, 3], [3, 2], 4, 1, 128, 64, kind, q_scale=0.0)
            ramp = torch.arange(p.cache.table.size(1) * 64, device="cuda").float() / 64
            for r in range(2):
                n = p.prefix[r] + p.win[r]
                g, t = p.cache.slots(r, 0, n)
                col = (ramp[:n] * slope + (12 if slope < 0 else 0))[:, None].expand(n, 1)
                if kind == "bf16":
                    p.cache.k[g, t, :, 5] = col.bfloat16()
                else:
                    p.cache.k.view(torch.uint8)[g, t, :, 5] = 0x38
                    p.cache.k_scale[g, :, t] = col
            p.q[:, :, 5] = 1000.0
            p.run(api).check()


def test_small_scale_zero_and_negative(api, dev):
    for scale in (0.0, -0.3, 2.0 ** -20):
        p = Problem(10, [200], [4], 4, 2, 64, 32, "bf16")
        p.scale = scale
        p.run(api).check()


def test_without_lse_and_again(api, dev):
    """No lse output; a second call gives the same bits."""
    p = Problem(11, [900, 12, 400], [9, 3, 1], 16, 2, 128, 64, "bf16").run(api, lse=False)
    assert bool((p.lse == 7).all())
    first = p.out.clone()
    p.run(api)
    assert torch.equal(first, p.out)
    p.check()


def test_bad_requests_leave_the_others(api, dev):
    for kind, dtype, page in (("bf16", "bf16", 16), ("f32", "f32", 16)):
        p = Problem(12, [40, 100, 33, 64], [4, 5, 3, 2], 4, 2, 64, page, kind, dtype=dtype)
        p.cache.table[1, 2] = p.cache.n_pages + 5
        p.run(api).check(skip=(1,))
        assert int(p.status) == api.STATUS_BAD_INDEX
        p = Problem(13, [40, 100, 33, 64], [4, 5, 3, 2], 4, 2, 64, page, kind, dtype=dtype)
        p.prefix_lens[2] = 10 ** 6
        p.run(api).check(skip=(2,))
        assert int(p.status) == api.STATUS_BAD_INDEX
        p = Problem(14, [40, 100, 33], [4, 32, 1], 4, 2, 64, page, kind, dtype=dtype)
        p.cu[2] += 1  # request 1 gets 33 rows, request 2 none
        p.run(api).check(skip=(1, 2))
        assert int(p.status) == api.STATUS_BAD_LEN


def test_pool_past_32_bits(api, dev):
    """Pages past 2^32 elements of the pool."""
    page, heads, D = 1024, 8, 128
    n = (1 << 32) // (page * heads * D) + 2
    p = Problem(15, [1500], [5], 16, heads, D, page, "e4m3", filled=False, pool=n)
    g = torch.Generator("cuda").manual_seed(1)
    p.cache.table[:] = torch.tensor([[n - 1, n - 2]], dtype=torch.int32)
    for t in (p.cache.k, p.cache.v):
        t.view(torch.uint8)[n - 2:] = torch.randint(0, 127, (2, page, heads, D), generator=g,
                                                    device="cuda", dtype=torch.uint8)
    p.run(api).check()


def test_on_a_side_stream_and_in_a_graph(api, dev):
    p = Problem(16, [300, 20], [5, 2], 8, 2, 128, 64, "bf16")
    ws = api.workspace(api.dspark_tree_attention_workspace_bytes(8, 128))
    kv = p.cache.kv()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()

    def call():
        api.dspark_tree_attention(p.q, kv, cu_seqlens=p.cu, prefix_lens=p.prefix_lens,
                                  scale=p.scale, out=p.out, lse=p.lse, workspace=ws, status=p.status)

    with torch.cuda.stream(side):
        call()
        side.synchronize()
        p.check()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
    # the captured call reads the lengths anew
    p.prefix = [123, 7]
    p.prefix_lens.copy_(torch.tensor(p.prefix, dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    p.check()


def test_argument_errors(api, dev):
    p = Problem(17, [30], [2], 4, 2, 64, 16, "bf16")
    ws = api.workspace(api.dspark_tree_attention_workspace_bytes(4, 64))
    ok = dict(cu_seqlens=p.cu, prefix_lens=p.prefix_lens, scale=1.0, out=p.out, workspace=ws,
              status=p.status)
    with pytest.raises(ValueError):
        api.dspark_tree_attention(p.q, p.cache.kv(), **{**ok, "out": p.out.float()})
    with pytest.raises(ValueError):
        api.dspark_tree_attention(p.q, p.cache.kv(), **{**ok, "cu_seqlens": p.cu[:1]})
    with pytest.raises(api.DsparkError):
        api.dspark_tree_attention(p.q, p.cache.kv(), **{**ok, "scale": math.nan})
    with pytest.raises(api.DsparkError):
        api.dspark_tree_attention(p.q, p.cache.kv(), **{**ok, "workspace": ws[:128]})
    with pytest.raises(api.DsparkError):
        api.dspark_tree_attention(p.q[:, :3], p.cache.kv(), **{**ok, "out": p.out[:, :3]})
    with pytest.raises(ValueError):
        api.dspark_tree_attention(p.q, p.cache.kv(), lse=p.lse[:1], **ok)
    assert int(p.status) == 0 and bool((p.out == 7).all())


# Decoding over the 8-bit cache, no more rows than requests (pad=0, or empty windows
# beside the longer ones), which takes a kernel of its own up to 8 heads a key head.
SINGLES = [
    dict(prefix=[0], win=[1], hq=1, hkv=1, D=64, page=16),
    dict(prefix=[1], win=[1], hq=8, hkv=1, D=128, page=64),
    dict(prefix=[0, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129], win=[1] * 11, hq=8, hkv=2, D=128, page=16),
    dict(prefix=[0, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129], win=[1] * 11, hq=5, hkv=1, D=64, page=48),
    # past the lengths at which every job stays whole
    dict(prefix=[700, 3, 512, 0, 1], win=[1] * 5, hq=16, hkv=2, D=128, page=256),
    dict(prefix=[30001], win=[1], hq=16, hkv=2, D=128, page=16),
    dict(prefix=[20000, 5, 9000], win=[1, 1, 1], hq=12, hkv=4, D=64, page=80),
    # longer windows beside empty ones; row tiles of one, two, four and eight tokens
    dict(prefix=[300, 7, 0, 1000, 9, 50], win=[4, 0, 1, 0, 0, 0], hq=8, hkv=1, D=128, page=32),
    dict(prefix=[640] + [33] * 40, win=[32] + [0] * 33 + [1] * 7, hq=8, hkv=2, D=128, page=64),
    dict(prefix=[63] + [33] * 40, win=[31] + [0] * 40, hq=6, hkv=3, D=64, page=64),
    dict(prefix=[14, 333, 1200], win=[3, 0, 0], hq=2, hkv=2, D=128, page=64),
    # more requests than a CTA has threads
    dict(prefix=[(37 * i) % 300 for i in range(700)], win=[i % 3 > 0 for i in range(700)], hq=4, hkv=2,
         D=64, page=64),
    dict(prefix=[(91 * i) % 900 for i in range(300)], win=[1] * 300, hq=8, hkv=1, D=128, page=16),
    # nine heads a key head: not this kernel
    dict(prefix=[700, 3], win=[1, 1], hq=9, hkv=1, D=128, page=64),
]


@pytest.mark.parametrize("i", range(len(SINGLES)))
@pytest.mark.parametrize("tree", [None, "orphans"])
def test_single_tokens_over_8_bits(api, dev, i, tree):
    shape = {**SINGLES[i], "win": [int(w) for w in SINGLES[i]["win"]]}
    p = Problem(300 + i, tree=tree, kind="e4m3", pad=0, **shape).run(api)
    p.check()
    assert int(p.status) == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_more_requests_than_threads(api, dev, kind):
    p = Problem(320, [(37 * i) % 200 for i in range(900)], [(i * 7) % 4 for i in range(900)], 4, 2, 64, 64,
                kind, tree="tree").run(api)
    p.check()
    assert int(p.status) == 0


@pytest.mark.parametrize("pad", [0, 9])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_odd_scales_and_unseen_values(api, dev, pad, bad):
    """Negative scales; scales and values that are not finite in places that a row
    does not see, in ones that it does, and past the requests' ends (pad=0: single
    tokens and empty windows)."""
    win = [3, 1, 1, 0, 0, 1] if pad == 0 else [3, 1, 1, 0, 2, 1]
    p = Problem(330, [37, 64, 5, 90, 20, 600], win, 8, 2, 128, 16, "e4m3", tree="orphans", pad=pad)
    c = p.cache
    used = torch.zeros((c.n_pages, 16), dtype=torch.bool, device="cuda")
    for r, (P, L) in enumerate(zip(p.prefix, p.win)):
        g, t = c.slots(r, 0, P + L)
        used[g, t] = True
    for t in (c.k, c.v):
        t.view(torch.uint8)[~used] = 0x7F
    for s in (c.k_scale, c.v_scale):
        s *= torch.where(torch.rand(s.shape, device="cuda") < 0.3, -1.0, 1.0)
        s.masked_fill_(~used[:, None, :], bad)
    c.put("v", 0, 37 + 1, bad)  # a token of the window that the rows after it do not see
    c.put("k", 0, 37 + 1, bad)
    c.put("v", 5, 17, math.nan)  # in a prefix
    p.run(api).check()
    assert int(p.status) == 0


@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_queries_of_wide_range(api, dev, kind, pad):
    """Queries whose elements differ by orders of magnitude, and rows of them that are
    tiny, huge, zero, infinite or NaN."""
    p = Problem(340, [130, 40, 77, 9, 21, 64], [1] * 6, 4, 2, 128, 64, kind, pad=pad)
    p.q[:6] *= 2.0 ** torch.randint(-9, 1, p.q[:6].shape, device="cuda")
    p.q[1] *= 2.0 ** -100
    p.q[2] *= 2.0 ** 7
    p.q[3] = 0
    p.q[4, 1, 7] = math.nan
    p.run(api).check(far_below=True)  # one-hot weights: dimensions where the one value is zero
    assert int(p.status) == 0


def test_bad_pages_of_single_tokens(api, dev):
    p = Problem(350, [40, 100, 33, 64], [1] * 4, 4, 2, 64, 16, "e4m3", pad=0)
    p.cache.table[1, 2] = p.cache.n_pages + 5
    p.run(api).check(skip=(1,))
    assert int(p.status) == api.STATUS_BAD_INDEX
    p = Problem(351, [40, 100, 33, 64], [1] * 4, 4, 2, 64, 16, "e4m3", pad=0)
    p.prefix_lens[2] = 10 ** 6
    p.run(api).check(skip=(2,))
    assert int(p.status) == api.STATUS_BAD_INDEX
