"""The two kernels of dspark_tree_attention over an 8-bit cache: eight query rows of a
kv head at once, or up to 128.  Which of them does a call is the library's choice; here
the second is asked for by scales that do not lie on 16 bytes, which the first does not
take, so that no choice of the library takes it out of its tests."""

import math

import pytest
import torch

import window_oracle as wo
from gpu_helpers import require_gpu
from test_gpu_attention import Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    require_gpu()
    from confidence_scheduled_speculative_gb300 import api
    return api


def _off_16_bytes(t):
    """The same tensor 4 bytes past a 16-byte boundary."""
    flat = torch.empty(t.numel() + 4, device=t.device, dtype=t.dtype)
    moved = flat[1:1 + t.numel()].view(t.shape)
    assert moved.data_ptr() % 16 == 4
    return moved.copy_(t)


class Wide(Problem):
    """A problem for the kernel of 128 rows."""

    def run(self, api, lse=True):
        c = self.cache
        if c.k_scale.data_ptr() % 16 == 0:
            c.k_scale, c.v_scale = _off_16_bytes(c.k_scale), _off_16_bytes(c.v_scale)
        return super().run(api, lse)


# ------------------------------------------------------------ which one

def _wide_did(api, shape):
    """Whether the bits of a call are those of the kernel of 128 rows."""
    a = Problem(600, kind="e4m3", **shape).run(api)
    b = Wide(600, kind="e4m3", **shape).run(api)
    a.check()
    b.check()
    return torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)


G4, G8 = dict(hq=8, hkv=2, D=128, page=64), dict(hq=16, hkv=2, D=128, page=64)


@pytest.mark.parametrize("wide,shape", [
    # long windows of two requests among slots without a row, one tree over a long prefix
    # beside single tokens, whatever the rows of the call have room for
    (True, dict(prefix=[3000, 2500] + [900] * 62, win=[32, 32] + [0] * 62, pad=0, **G8)),
    (True, dict(prefix=[40000] + [70] * 63, win=[32] + [1] * 63, pad=33, **G4)),
    (True, dict(prefix=[3000] * 8 + [9] * 24, win=[8] * 8 + [0] * 24, pad=0, **G4)),
    (True, dict(prefix=[3000] * 4, win=[32] * 4, pad=64, **G4)),
    # single tokens, beside slots without one and beside a long window over nothing much
    (False, dict(prefix=[3000] * 20, win=[1] * 20, pad=0, **G4)),
    (False, dict(prefix=[3000] * 20, win=[1] * 20, pad=400, **G4)),
    (False, dict(prefix=[3000] * 9 + [50] * 80, win=[1] * 9 + [0] * 80, pad=3, **G8)),
    (False, dict(prefix=[30000, 0], win=[1, 32], pad=0, **G4)),
])
def test_the_work_decides(api, wide, shape):
    """Passes over the long prefixes decide, not rows over requests."""
    assert _wide_did(api, shape) == wide


# ------------------------------------------------- the one of 128 rows

SHAPES = [
    dict(prefix=[0], win=[1], hq=1, hkv=1, D=64, page=16),
    dict(prefix=[0, 5, 0, 16], win=[1, 1, 3, 1], hq=8, hkv=2, D=128, page=16),
    # lengths around tile and page ends, windows of zero
    dict(prefix=[63, 64, 65, 127, 128, 1, 0], win=[1, 1, 1, 1, 17, 0, 0], hq=8, hkv=1, D=128, page=64),
    dict(prefix=[15, 16, 17, 31, 48, 200], win=[1, 2, 1, 9, 32, 5], hq=12, hkv=4, D=64, page=48),
    # 64 rows and fewer, then more, of one request after another; one row past 64 and 128
    dict(prefix=[700, 90, 1300], win=[32, 16, 17], hq=8, hkv=2, D=64, page=64),
    dict(prefix=[129, 4000], win=[13, 26], hq=5, hkv=1, D=128, page=32),
    dict(prefix=[511], win=[32], hq=32, hkv=2, D=64, page=48),
    dict(prefix=[300, 9], win=[3, 32], hq=86, hkv=2, D=128, page=16),  # 43 heads a kv head
    # many requests, more than a CTA has threads; jobs split over many CTAs
    dict(prefix=[(37 * i) % 500 for i in range(70)], win=[i % 6 for i in range(70)], hq=4, hkv=2, D=128, page=64),
    dict(prefix=[(37 * i) % 200 for i in range(900)], win=[(i * 7) % 4 for i in range(900)], hq=4, hkv=2,
         D=64, page=64),
    dict(prefix=[30001], win=[1], hq=16, hkv=2, D=128, page=16),
    dict(prefix=[20000, 3], win=[17, 32], hq=8, hkv=1, D=64, page=128),
]


@pytest.mark.parametrize("i", range(len(SHAPES)))
@pytest.mark.parametrize("tree", [None, "orphans"])
def test_wide(api, i, tree):
    p = Wide(620 + i, tree=tree, kind="e4m3", **SHAPES[i]).run(api)
    p.check()
    assert int(p.status) == 0
    out, lse = p.out.clone(), p.lse.clone()
    p.run(api)
    assert torch.equal(out, p.out) and torch.equal(lse, p.lse)  # a call repeated


KERNELS = [pytest.param(Problem, [1, 1, 1, 0, 1, 1], id="few"), pytest.param(Wide, [3, 1, 32, 0, 2, 1], id="wide")]


@pytest.mark.parametrize("kernel,win", KERNELS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, None])
def test_odd_scales(api, kernel, win, D, bad):
    """Negative scales of keys and values (bad=None: nothing else, in prefixes as in
    windows); scales and codes that are not finite past the ends, in pages of no
    request, in tokens that a row does not see, and in a prefix."""
    p = kernel(640, [137, 264, 5, 90, 20, 600], win, 8, 2, D, 16, "e4m3", tree="orphans", pad=0)
    c = p.cache
    for s in (c.k_scale, c.v_scale):
        s *= torch.where(torch.rand(s.shape, device="cuda") < 0.3, -1.0, 1.0)
    if bad is not None:
        used = torch.zeros((c.n_pages, 16), dtype=torch.bool, device="cuda")
        for r, (P, L) in enumerate(zip(p.prefix, p.win)):
            g, t = c.slots(r, 0, P + L)
            used[g, t] = True
        for t in (c.k, c.v):
            t.view(torch.uint8)[~used] = 0x7F
        for s in (c.k_scale, c.v_scale):
            s.masked_fill_(~used[:, None, :], bad)
        for which in "kv":
            if win[0] > 1:
                c.put(which, 0, 137 + 1, bad)  # which the rows after it do not see
            if win[2] > 1:
                c.put(which, 2, 5 + 7, bad)
        c.put("v", 5, 17, math.nan)
    p.run(api).check()
    assert int(p.status) == 0


@pytest.mark.parametrize("kernel,win", [pytest.param(Problem, [1, 1], id="few"), pytest.param(Wide, [3, 20], id="wide")])
@pytest.mark.parametrize("slope", [1, -1])
def test_a_maximum_that_moves(api, kernel, win, slope):
    """Scores of thousands that rise, or fall, along the prefix."""
    p = kernel(650, [700, 3], win, 4, 1, 128, 64, "e4m3", q_scale=0.0)
    ramp = torch.arange(p.cache.table.size(1) * 64, device="cuda").float() / 64
    for r in range(2):
        n = p.prefix[r] + p.win[r]
        g, t = p.cache.slots(r, 0, n)
        p.cache.k.view(torch.uint8)[g, t, :, 5] = 0x38
        p.cache.k_scale[g, :, t] = (ramp[:n] * slope + (12 if slope < 0 else 0))[:, None]
    p.q[:, :, 5] = 1000.0
    p.run(api).check()


@pytest.mark.parametrize("kernel,win", [pytest.param(Problem, [1, 1], id="few"), pytest.param(Wide, [4, 32], id="wide")])
@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0 ** -20])
def test_scales_of_the_scores(api, kernel, win, scale):
    p = kernel(660, [200, 70], win, 4, 2, 64, 32, "e4m3")
    p.scale = scale
    p.run(api).check()


@pytest.mark.parametrize("kernel,win", [pytest.param(Problem, [1] * 4, id="few"), pytest.param(Wide, [4, 32, 3, 2], id="wide")])
def test_bad_requests_leave_the_others(api, kernel, win):
    def problem(seed):
        return kernel(seed, [40, 100, 33, 64], win, 4, 2, 64, 16, "e4m3")
    p = problem(670)
    p.cache.table[1, 2] = p.cache.n_pages + 5
    p.run(api).check(skip=(1,))
    assert int(p.status) == api.STATUS_BAD_INDEX
    p = problem(671)
    p.cache.table[2, 0] = -1
    p.prefix_lens[3] = -7
    p.run(api).check(skip=(2, 3))
    assert int(p.status) == api.STATUS_BAD_INDEX
    p = problem(672)
    p.prefix_lens[2] = 10 ** 6
    p.run(api).check(skip=(2,))
    assert int(p.status) == api.STATUS_BAD_INDEX
    if win[1] == 32:
        p = problem(673)
        p.cu[2] += 1  # 33 rows, and the next request two
        p.run(api).check(skip=(1, 2))
        assert int(p.status) == api.STATUS_BAD_LEN


def test_wide_pool_past_32_bits(api):
    """Pages past 2^32 elements of the pool."""
    page, heads, D = 1024, 8, 128
    n = (1 << 32) // (page * heads * D) + 2
    p = Wide(680, [1500], [17], 16, heads, D, page, "e4m3", filled=False, pool=n)
    g = torch.Generator("cuda").manual_seed(1)
    p.cache.table[:] = torch.tensor([[n - 1, n - 2]], dtype=torch.int32)
    for t in (p.cache.k, p.cache.v):
        t.view(torch.uint8)[n - 2:] = torch.randint(0, 127, (2, page, heads, D), generator=g,
                                                    device="cuda", dtype=torch.uint8)
    p.run(api).check()
    assert int(p.status) == 0


# Over E4M3 the kernel of 128 rows takes a query as two E4M3 numbers, hi + lo, after a
# power of two has brought the row's largest element to 128..256.  E4M3 has four digits
# and a smallest step of 2^-9: a bfloat16 of eight digits is hi + lo exactly while its
# last digit is 2^-9 or more, which holds from 2^-2 on, 2^-9 of a largest element of
# 128.  Below, half a step is lost: 2^-10, at most 2^-17 of the largest.

def test_query_split_by_its_formats():
    """That bound, over every bfloat16 from 256 down, against the largest element of the
    range, by rounding to E4M3 as torch does."""
    bits = torch.arange(0, 0x4380, dtype=torch.int32)  # 0 .. 256
    x = (bits << 16).view(torch.float32)
    hi = x.to(torch.float8_e4m3fn).float()
    lo = (x - hi).to(torch.float8_e4m3fn).float()
    off = (x.double() - hi.double() - lo.double()).abs()
    assert not bool(off[x >= 128 * 2.0 ** -9].any())
    assert 2.0 ** -18 < float(off.max()) / 128 <= 2.0 ** -17


class Split(Wide):
    """With what the queries' parts lose."""

    def check(self):
        lo = 0
        for r, (P, L) in enumerate(zip(self.prefix, self.win)):
            if not L:
                continue
            q = self.q[lo:lo + L]
            o, lse, tol, lse_tol, o_abs = wo.attention(q, self.cache, r, P, L, self.bits[r], self.scale)
            # each small element's loss times the largest key element it may meet
            size = torch.nan_to_num(q.double().abs())
            most = size.amax(-1, keepdim=True)
            lost = torch.where(size < most * 2.0 ** -9, most * 2.0 ** -17, 0.0)
            k = self.cache.values("k", r, 0, P + L).abs().permute(1, 2, 0)  # [kv heads, D, n]
            k = k.repeat_interleave(self.hq // k.size(0), 0)
            e = torch.einsum("lhd,hdn->lhn", lost, k).amax(-1) * abs(self.scale)
            got, got_lse = self.out[lo:lo + L].double(), self.lse[lo:lo + L].double()
            assert torch.equal(torch.isnan(got), torch.isnan(o)), r
            # (weights off by exp(+-e), their sum likewise; weights as halves, far below
            # the largest of all; a position's weight is one step off at the least)
            bound = (tol + (self.unit() + torch.expm1(2 * e)[..., None]) * o_abs) * (1 + wo.BF16) \
                + wo.BF16 * o.abs() + 1e-38 + self.smallest_weight(r, P + L)
            off = ((got - o).abs() - bound)[torch.isfinite(o)]
            assert float(off.max()) <= 0, (r, float(off.max()))
            off = ((got_lse - lse).abs() - lse_tol - e)[torch.isfinite(lse)]
            assert float(off.max()) <= 0, (r, float(off.max()))
            lo += L


@pytest.mark.parametrize("D", [64, 128])
def test_wide_queries_of_wide_range(api, D):
    """Queries whose elements differ by up to 2^16, and rows that are tiny, huge, zero or
    hold a NaN."""
    win = [1, 5, 17, 2, 3, 32]
    p = Split(690, [130, 40, 77, 9, 21, 64], win, 4, 2, D, 64, "e4m3")
    p.q *= 2.0 ** torch.randint(-16, 1, p.q.shape, device="cuda")
    p.q[1] *= 2.0 ** -100
    p.q[7] *= 2.0 ** 5
    p.q[9] = 0
    p.q[24, 1, 7] = math.nan
    p.run(api).check()
    assert int(p.status) == 0


@pytest.mark.parametrize("kernel", [Problem, Wide])
def test_one_captured_call_serves_both_kernels(api, kernel):
    """A graph holds both kernels; the lengths at each replay choose anew."""
    p = kernel(700, [900] * 12, [3] * 12, 8, 1, 128, 64, "e4m3")
    if kernel is Wide:
        p.run(api)  # moves the scales
    ws = api.workspace(api.dspark_tree_attention_workspace_bytes(p.hq, p.D))
    kv, graph = p.cache.kv(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.dspark_tree_attention(p.q, kv, cu_seqlens=p.cu, prefix_lens=p.prefix_lens, scale=p.scale,
                                  out=p.out, lse=p.lse, workspace=ws, status=p.status)
    for win, prefix in (([1] * 12, [870 + i for i in range(12)]), ([32] + [0] * 10 + [4], [870] * 12),
                        ([3] * 12, [5] * 12), ([0] * 11 + [1], [900] * 12), ([0] * 12, [0] * 12),
                        ([32, 2, 2], [0, 850, 850])):
        win, prefix = win + [0] * (12 - len(win)), prefix + [0] * (12 - len(prefix))
        p.win, p.prefix, p.rows = win, prefix, sum(win)
        p.bits = [wo.chain_bits(w) for w in win]
        p.cu.copy_(torch.tensor([0] + win).cumsum(0))
        p.prefix_lens.copy_(torch.tensor(prefix))
        p.out.fill_(7.0)
        p.lse.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        p.check()
    assert int(p.status) == 0
