"""Causal attention of ragged prompts (dspark_prompt_attention) against its 64-bit
definition."""

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


class Problem:
    def __init__(self, seed, lens, hq, hkv=None, K=128, S=64, V=128, dtype="bf16", pad=3, together=True):
        """lens: (queries, keys) of each request."""
        g = torch.Generator("cuda").manual_seed(seed)
        hkv = hkv or hq
        dt = self.dtype = wo.DTYPES[dtype]
        self.lens, self.S = lens, S
        n, m = (sum(x) for x in zip(*lens))
        self.n = n
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(dt)
        wide = rnd(n + pad, hq + 1, K + S) * 2  # queries beside other columns, where `together`
        self.q = wide[:, :hq] if together else wide[:, :hq].contiguous()
        if together:  # a head's keys and values side by side, as one projection leaves them
            kv = rnd(m + pad, hkv, K + V)
            self.k, self.v = kv[..., :K], kv[..., K:]
        else:
            self.k, self.v = rnd(m + pad, hkv, K), rnd(m + pad, hkv, V)
        self.k_shared = rnd(m + pad, S + 8)[:, :S] if S else None
        self.scale = (K + S) ** -0.5
        self.cu = torch.tensor([0] + [a for a, _ in lens], device="cuda").cumsum(0).int()
        self.cu_k = torch.tensor([0] + [b for _, b in lens], device="cuda").cumsum(0).int()
        self.out = torch.full((n + pad, hq, V), 7.0, device="cuda", dtype=dt)
        self.lse = torch.full((n + pad, hq), 7.0, device="cuda")
        self.status = torch.zeros(1, **I32)
        self.unit = wo.BF16 if (dtype, K, V) == ("bf16", 128, 128) and S in (0, 64) else 0.0

    def call(self, api, lse=True):
        api.dspark_prompt_attention(self.q, self.k, self.v, k_shared=self.k_shared, cu_seqlens=self.cu,
                                    cu_keys=self.cu_k, scale=self.scale, out=self.out,
                                    lse=self.lse if lse else None, status=self.status)

    def run(self, api, **kw):
        self.call(api, **kw)
        torch.cuda.synchronize()
        return self

    def check(self, skip=()):
        cu, cu_k = self.cu.tolist(), self.cu_k.tolist()
        for r, (n, m) in enumerate(self.lens):
            if not n or r in skip:
                continue
            a, b = slice(cu[r], cu[r] + n), slice(cu_k[r], cu_k[r] + m)
            want = lo.prompt(self.q[a], self.k[b], self.k_shared[b] if self.S else None, self.v[b], self.scale)
            lo.compare(self.out[a], self.lse[a], want, self.unit, self.dtype, r)
        assert bool((self.out[self.n:] == 7).all()) and bool((self.lse[self.n:] == 7).all())
        return self


SHAPES = [
    dict(lens=[(1, 1)], hq=1),
    dict(lens=[(1, 1), (2, 2), (3, 5), (0, 7), (0, 0), (4, 4)], hq=3),
    # around the ends of tiles, with and without keys before the queries
    dict(lens=[(63, 63), (64, 64), (65, 65), (127, 130), (128, 128), (129, 257)], hq=2),
    dict(lens=[(255, 255), (256, 256), (257, 300), (1, 1000), (511, 513)], hq=2),
    dict(lens=[(700, 1900), (33, 33)], hq=5, together=False),
    # fewer keys than queries: the first rows see nothing
    dict(lens=[(5, 2), (4, 0), (300, 170), (260, 3), (2, 2)], hq=2),
    # heads that share keys, keys without a shared part
    dict(lens=[(300, 420), (17, 17)], hq=8, hkv=2),
    dict(lens=[(300, 420), (17, 17), (129, 640)], hq=6, hkv=3, S=0),
    dict(lens=[(1 + i % 7, 1 + (11 * i) % 40 + i % 7) for i in range(150)], hq=2),
    # in 32 bits throughout
    dict(lens=[(70, 90), (3, 1)], hq=2, dtype="f32"),
    dict(lens=[(70, 90), (3, 3)], hq=4, hkv=2, K=33, S=7, V=50),
    dict(lens=[(40, 41)], hq=2, K=256, S=256, V=256, dtype="f32"),
    dict(lens=[(40, 41)], hq=2, K=1, S=0, V=1),
    dict(lens=[(40, 41)], hq=2, K=64, S=0, V=64),
]


@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_prompt(api, i):
    p = Problem(300 + i, **SHAPES[i]).run(api).check()
    assert int(p.status) == 0


@pytest.mark.parametrize("shape", [dict(hq=2), dict(hq=4, hkv=2, S=0), dict(hq=2, K=24, S=8, V=40)])
def test_unseen_keys_have_no_effect(api, shape):
    """NaN and infinities in other requests' keys and behind the last, and in keys that
    a prompt's first rows do not see; the rows that do see them get what the formula gives."""
    for value in (math.nan, math.inf, -math.inf):
        p = Problem(320, [(140, 150), (200, 333), (9, 9)], **shape)
        last = int(p.cu_k[-1])
        p.k[last:], p.v[last:] = value, value
        p.k[150:483], p.v[150:483] = value, value
        if p.S:
            p.k_shared[last:] = value
        p.run(api).check(skip=(1,))
        assert int(p.status) == 0
        # a key in the middle of a prompt: rows before it are as without it
        p = Problem(321, [(300, 310), (40, 40)], **shape)
        at = 10 + 130
        p.v[at] = value
        p.run(api).check()
        p.k[at] = value
        p.v[at] = 1.0
        p.run(api)
        want = lo.prompt(p.q[:130], p.k[:140], p.k_shared[:140] if p.S else None, p.v[:140], p.scale)
        lo.compare(p.out[:130], p.lse[:130], want, p.unit, p.dtype, value)


def test_scores_far_apart(api):
    for scale in (30.0, 0.0, -1.0, 1e-30):
        p = Problem(330, [(200, 260), (70, 70)], hq=2)
        p.scale = scale if scale <= 0 or scale < 1e-20 else p.scale * scale
        p.run(api).check()


@pytest.mark.parametrize("shape", [dict(hq=2), dict(hq=2, K=24, S=8, V=40)])
def test_bad_ranges_do_not_disturb_others(api, shape):
    p = Problem(340, [(70, 80), (300, 310), (20, 20)], **shape)
    p.cu_k[3] = 10 ** 6  # the last request's keys end behind the buffer
    p.run(api).check(skip=(2,))
    assert int(p.status) == api.STATUS_BAD_LEN
    p = Problem(341, [(70, 80), (300, 310)], **shape)
    p.cu[2] = p.q.size(0) + 9
    p.n = p.q.size(0)
    p.run(api).check(skip=(1,))
    assert int(p.status) == api.STATUS_BAD_LEN


def test_more_requests_than_threads(api):
    p = Problem(345, [((7 * i) % 5, (7 * i) % 5 + (3 * i) % 20) for i in range(700)] + [(600, 700)], hq=2)
    p.run(api).check()
    assert int(p.status) == 0


@pytest.mark.parametrize("shape", [dict(hq=3), dict(hq=4, hkv=2, S=0)])
def test_short_requests_beside_long_ones(api, shape):
    """Mostly single tokens, and requests on both sides of what counts as short."""
    lens = [(1, 1)] * 150 + [(22, 23), (23, 23), (16, 32), (1, 512), (1, 513), (0, 3), (600, 700), (40, 10), (2, 257)]
    p = Problem(348, lens + [(1, 2)] * 150, **shape).run(api).check()
    assert int(p.status) == 0
    p.cu[5], p.cu_k[8] = p.n + 100, 1 << 30  # two ranges that end outside, two that begin there
    p.out.fill_(7), p.lse.fill_(7)
    p.run(api)
    assert int(p.status) == api.STATUS_BAD_LEN


def test_two_at_once(api):
    """Calls on two streams."""
    two = [Problem(346, [(300, 900), (5, 5)], hq=6).run(api).check(), Problem(347, [(513, 513)], hq=8, S=0).run(api).check()]
    first = [(p.out.clone(), p.lse.clone()) for p in two]
    streams = [torch.cuda.Stream() for _ in two]
    for p in two:
        p.out.fill_(7), p.lse.fill_(7)
    torch.cuda.synchronize()
    for _ in range(5):
        for p, s in zip(two, streams):
            with torch.cuda.stream(s):
                p.call(api)
    torch.cuda.synchronize()
    for p, (out, lse) in zip(two, first):
        assert torch.equal(p.out, out) and torch.equal(p.lse, lse) and int(p.status) == 0


def test_repeated_and_captured(api):
    p = Problem(350, [(300, 700), (129, 129)], hq=4).run(api).check()
    first = p.out.clone()
    p.out.fill_(7)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.call(api)
    for _ in range(2):
        p.out.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(p.out, first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    p.out.fill_(7)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        p.call(api, lse=False)
    side.synchronize()
    assert torch.equal(p.out, first)


def test_refusals(api):
    p = Problem(360, [(5, 6)], hq=2)
    kw = dict(cu_seqlens=p.cu, cu_keys=p.cu_k, scale=1.0, status=p.status)
    with pytest.raises(ValueError, match="q"):
        api.dspark_prompt_attention(p.q, p.k, p.v, out=p.out, **kw)  # no shared part
    with pytest.raises(ValueError, match="out"):
        api.dspark_prompt_attention(p.q, p.k, p.v, k_shared=p.k_shared, out=p.out[..., :64], **kw)
    with pytest.raises(ValueError, match="v"):
        api.dspark_prompt_attention(p.q, p.k, p.v[:2], k_shared=p.k_shared, out=p.out, **kw)
    with pytest.raises(api.DsparkError):
        api.dspark_prompt_attention(p.q, p.k, p.v, k_shared=p.k_shared, out=p.out, **{**kw, "scale": math.nan})
    both = torch.zeros((8, 2, 192), device="cuda", dtype=torch.bfloat16)
    over = both.view(8, -1)[:, :256].unflatten(1, (2, 128))
    with pytest.raises(api.DsparkError):
        api.dspark_prompt_attention(both, p.k, p.v, k_shared=p.k_shared, out=over, **kw)


@pytest.mark.parametrize("shape", [dict(hq=2), dict(hq=4, hkv=2, S=0), dict(hq=2, K=24, S=8, V=40)])
def test_seen_infinite_elements(api, shape):
    """Infinite values under a weight (infinite too), and under the weight 0 of a score of
    -inf (NaN), among keys that all rows see and among those that some do."""
    for value in (math.inf, -math.inf):
        for at in (4, 300):
            p = Problem(322, [(300, 510), (40, 40)], **shape)
            p.v[at, :, 5] = value
            p.v[at + 64, :, p.v.size(2) - 1] = value
            p.k[at, :, 7] = value
            p.run(api).check()
            assert bool(p.out.isnan().any()) and bool(p.out.isinf().any()) and int(p.status) == 0


def test_output_beside_keys_and_values(api):
    """In the same rows of one buffer, sharing no element; over a part of them it is refused."""
    p = Problem(361, [(40, 40), (7, 7)], hq=2, pad=0).run(api)
    first, n = p.out.clone(), p.k.size(0)
    rows = torch.zeros((n, 2 * 256 + 64 + 256), device="cuda", dtype=torch.bfloat16)
    heads = rows[:, :512].unflatten(1, (2, 256))
    heads[..., :128], heads[..., 128:], rows[:, 512:576] = p.k, p.v, p.k_shared
    kept = rows[:, :576].clone()
    p.k, p.v, p.k_shared = heads[..., :128], heads[..., 128:], rows[:, 512:576]
    p.out = rows[:, 576:].unflatten(1, (2, 128))
    p.run(api)
    assert torch.equal(p.out, first) and torch.equal(rows[:, :576], kept) and int(p.status) == 0
    for at in (0, 128, 400, 575):  # over keys, values, both, the shared part
        p.out = rows[:, at:at + 256].unflatten(1, (2, 128))
        with pytest.raises(api.DsparkError):
            p.run(api)
    assert torch.equal(rows[:, :576], kept)


@pytest.mark.parametrize("shape", [dict(hq=3), dict(hq=4, hkv=2, S=0)])
@pytest.mark.parametrize("last", [(3, 3), (600, 700)])
@pytest.mark.parametrize("which", ["rows", "keys"])
def test_bad_ranges_beside_short_requests(api, shape, last, which):
    """Where both kernels run: a last range, short or long, that ends outside the rows or the
    keys leaves the other requests of either kernel as they are."""
    lens = [(1, 1)] * 150 + [(22, 23), (300, 400), (16, 33), (1, 513), (0, 3)] + [(1, 2)] * 150 + [last]
    p = Problem(349, lens, **shape)
    assert (p.q.size(0) + p.k.size(0)) // 46 < len(lens)
    if which == "rows":
        p.cu[-1] = p.q.size(0) + 9
        p.n = p.q.size(0)
    else:
        p.cu_k[-1] = p.k.size(0) + 9
    p.run(api).check(skip=(len(lens) - 1,))
    assert int(p.status) == api.STATUS_BAD_LEN
