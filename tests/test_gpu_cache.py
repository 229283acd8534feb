"""Norms and rotation of queries and keys, the quantising cache write and its
reading back (dspark_qk_norm_rope, dspark_kv_append, dspark_kv_read) against
their 64-bit definitions."""

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


def _angles(n, rope):
    a = torch.arange(n, device="cuda").double()[:, None] * 10000.0 ** (
        -torch.arange(0, rope, 2, device="cuda").double() / rope)
    return torch.cat([a.cos(), a.sin()], 1).float()


def _status(dev):
    return torch.zeros(1, dtype=torch.int32, device=dev)


def _close(got, want, tol, unit):
    """Within the 32-bit error and the one rounding to the output's type."""
    got = got.double()
    off = (got - want).abs() - (tol * (1 + unit) + unit * want.abs() + 2.0 ** -133)
    assert bool((off <= 0).all()), float(off.max())


SHAPES = [  # rows, hq, hkv, D, rope, interleaved, dtype, weights
    (1, 1, 1, 2, 2, False, "f32", "qk"),
    (1, 8, 2, 64, 64, False, "bf16", "qk"),
    (5, 3, 1, 80, 64, True, "f32", "qk"),
    (7, 5, 5, 80, 80, False, "bf16", "q"),
    (33, 64, 8, 128, 128, False, "bf16", "qk"),
    (33, 7, 1, 128, 64, True, "bf16", "k"),
    (12, 4, 2, 256, 128, False, "f32", "qk"),
    (9, 2, 2, 96, 96, True, "bf16", ""),
    (9, 6, 3, 34, 18, False, "bf16", "qk"),   # odd sizes: the any-layout kernel
    (9, 6, 3, 254, 254, True, "f32", "qk"),
    (4, 2, 1, 128, 0, False, "bf16", "qk"),
    (2049, 2, 1, 64, 32, False, "bf16", "qk"),
]


@pytest.mark.parametrize("rows,hq,hkv,D,rope,inter,dtype,weights", SHAPES)
@pytest.mark.parametrize("in_place", [False, True])
def test_norm_rope(api, dev, rows, hq, hkv, D, rope, inter, dtype, weights, in_place):
    g = torch.Generator("cuda").manual_seed(rows * 1000 + D)
    dt = wo.DTYPES[dtype]
    qkv = (torch.randn((rows + 3, hq + hkv, D), generator=g, device=dev) * 1.7).to(dt)
    q, k = qkv[:, :hq], qkv[:, hq:]
    w = {n: (1 + 0.3 * torch.randn(D, generator=g, device=dev)).to(dt) if n in weights else None
         for n in "qk"}
    table = _angles(300, rope) if rope else None
    pos = torch.randint(0, 300, (rows + 3,), generator=g, device=dev).int()
    totals = torch.tensor([rows, rows + 3], dtype=torch.int32, device=dev)
    want = {n: wo.norm_rope(t, w[n], 1e-5, table, pos, inter) for n, t in (("q", q), ("k", k))}
    before = qkv.clone()
    out = {"q": q, "k": k} if in_place else {n: torch.full_like(t, 7.0).contiguous()
                                            for n, t in (("q", q), ("k", k))}
    st = _status(dev)
    api.dspark_qk_norm_rope(q, k, pos=pos, totals=totals, q_weight=w["q"], k_weight=w["k"],
                            eps=1e-5, cos_sin=table, interleaved=inter, q_out=out["q"],
                            k_out=out["k"], status=st)
    for n in "qk":
        y, tol = want[n]
        _close(out[n][:rows], y[:rows], tol[:rows], wo.out_unit(dt))
    if in_place:
        assert torch.equal(qkv[rows:], before[rows:])
    else:
        assert bool((out["q"][rows:] == 7).all()) and bool((out["k"][rows:] == 7).all())
        assert torch.equal(qkv, before)
    assert int(st) == 0


def test_norm_rope_one_side_and_bad_positions(api, dev):
    g = torch.Generator("cuda").manual_seed(1)
    q = torch.randn((6, 4, 64), generator=g, device=dev)
    table = _angles(10, 64)
    pos = torch.tensor([0, 9, 10, -1, 3, 2 ** 31 - 1], dtype=torch.int32, device=dev)
    y, tol = wo.norm_rope(q, None, 0.0, table, pos.clamp(0, 9), False)
    out, st = torch.full_like(q, 5.0), _status(dev)
    api.dspark_qk_norm_rope(q, None, pos=pos, cos_sin=table, q_out=out, status=st)
    good = [0, 1, 4]
    _close(out[good], y[good], tol[good], wo.U32)
    assert bool((out[[2, 3, 5]] == 5).all())
    assert int(st) == api.STATUS_BAD_INDEX


CACHES = [  # kind, layout, page, D, dtype of the rows
    ("bf16", "tokens", 16, 64, "bf16"), ("bf16", "heads", 64, 128, "bf16"),
    ("e4m3", "tokens", 64, 128, "bf16"), ("e4m3", "heads", 16, 64, "f32"),
    ("e4m3", "tokens", 5, 80, "bf16"), ("f32", "tokens", 7, 128, "f32"),
    ("f32", "heads", 32, 64, "bf16"), ("bf16", "tokens", 1, 256, "f32"),
    ("e4m3", "heads", 3, 34, "f32"), ("bf16", "tokens", 24, 18, "bf16"),
]


def _check_stored(cache, which, r, p, y, tol):
    """Entries of positions p (a range) against 64-bit values y [n, heads, D]."""
    page, tok = cache.slots(r, p[0], p[1])
    t = (cache.k if which == "k" else cache.v)
    if cache.kind != "e4m3":
        _close(t[page, tok], y, tol, wo.out_unit(wo.DTYPES[cache.kind]))
        return
    s = (cache.k_scale if which == "k" else cache.v_scale)[page, :, tok].double()
    most = y.abs().amax(-1)
    want = (most / 448).clamp(min=2.0 ** -100)
    assert bool(((s - want).abs() <= (tol.amax(-1) / 448 + 2 * wo.U32 * want)).all())
    x = y / s[..., None]
    off = (wo.e4m3_values(t.view(torch.uint8)[page, tok]) - x).abs()
    # the nearest code, save where the 32-bit error moves x across a midpoint
    slack = tol / s[..., None] + 4 * wo.U32 * x.abs()
    assert bool((off <= wo.e4m3_step(x) / 2 + 2 * slack).all())


@pytest.mark.parametrize("kind,layout,page,D,dtype", CACHES)
@pytest.mark.parametrize("tree", [False, True])
def test_append_then_read(api, dev, kind, layout, page, D, dtype, tree):
    gen = torch.Generator().manual_seed(D + page)
    g = torch.Generator("cuda").manual_seed(D)
    hq, hkv = 6, 2
    prefix, win = [0, 1, page, 40, 2 * page + 1], [1, 9, 0, 32, 3]
    rows, pad = sum(win), 5
    cache = wo.Cache(gen, kind, [p + w for p, w in zip(prefix, win)], hkv, D, page, layout,
                     filled=False)
    dt = wo.DTYPES[dtype]
    qkv = torch.randn((rows + pad, hq + 2 * hkv, D), generator=g, device=dev).to(dt)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    req = torch.tensor([r for r, w in enumerate(win) for _ in range(w)] + [-1] * pad,
                       dtype=torch.int32, device=dev)
    at = torch.tensor([p + j for p, w in zip(prefix, win) for j in range(w)] + [0] * pad,
                      dtype=torch.int32, device=dev)
    # a tree's nodes rotate by depth, which is not their place in the window
    pos = torch.where(req >= 0, at // 2, 0) if tree else at
    weight = (1 + 0.2 * torch.randn(D, generator=g, device=dev)).to(dt)
    rope = D // 2 if D % 4 == 0 else D
    table = _angles(200, rope)
    q_out, st = torch.zeros((rows + pad, hq, D), device=dev, dtype=dt), _status(dev)
    api.dspark_kv_append(k, v, cache.kv(), q=q, q_out=q_out, req=req, pos=pos,
                         cache_pos=at if tree else None, q_weight=weight, k_weight=weight,
                         eps=1e-6, cos_sin=table, status=st)
    y, tol = wo.norm_rope(q[:rows], weight, 1e-6, table, pos[:rows], False)
    _close(q_out[:rows], y, tol, wo.out_unit(dt))
    assert not bool(q_out[rows:].any())
    y, tol = wo.norm_rope(k[:rows], weight, 1e-6, table, pos[:rows], False)
    lo = 0
    for r, (p, w) in enumerate(zip(prefix, win)):
        if w:
            _check_stored(cache, "k", r, (p, p + w), y[lo:lo + w], tol[lo:lo + w])
            x = v[lo:lo + w].double()
            _check_stored(cache, "v", r, (p, p + w), x, torch.zeros_like(x))
        lo += w
    assert int(st) == 0
    # back as rows, in both types: what the entries stand for, rounded once
    cu = torch.tensor([0] + win, device=dev).cumsum(0).int()
    start = torch.tensor(prefix, dtype=torch.int32, device=dev)
    for out in ("bf16", "f32"):
        ko = torch.full((rows + 2, hkv, D), 3.0, device=dev, dtype=wo.DTYPES[out])
        vo = ko.clone()
        api.dspark_kv_read(cache.kv(), start=start, cu_rows=cu, k_out=ko, v_out=vo, status=st)
        lo = 0
        for r, (p, w) in enumerate(zip(prefix, win)):
            for t, n in ((ko, "k"), (vo, "v")):
                if w:
                    x = cache.values(n, r, p, p + w)
                    _close(t[lo:lo + w], x, wo.U32 * x.abs(), wo.out_unit(wo.DTYPES[out]))
            lo += w
        assert bool((ko[rows:] == 3).all()) and bool((vo[rows:] == 3).all())
    assert int(st) == 0


def test_append_writes_only_its_slots(api, dev):
    """Every entry and scale outside the rows' slots keeps its bits; a strided
    pool (two layers interleaved) included."""
    gen = torch.Generator().manual_seed(3)
    for kind in ("bf16", "e4m3"):
        cache = wo.Cache(gen, kind, [70, 33], 2, 64, 16, scale=1.0)
        both = torch.zeros((cache.n_pages, 2, 16, 2, 64), device=dev, dtype=torch.uint8
                           if kind == "e4m3" else torch.bfloat16)
        if kind == "e4m3":
            both = both.view(torch.float8_e4m3fn)
        cache.k, other = both[:, 0], both[:, 1]
        v_both = both.clone()
        cache.v = v_both[:, 0]
        req = torch.tensor([0, 1, 1], dtype=torch.int32, device=dev)
        pos = torch.tensor([69, 0, 32], dtype=torch.int32, device=dev)
        k = torch.ones((3, 2, 64), device=dev, dtype=torch.bfloat16)
        before = [None if t is None else t.clone() for t in (cache.k_scale, cache.v_scale)]
        st = _status(dev)
        api.dspark_kv_append(k, 2 * k, cache.kv(), req=req, pos=pos, status=st)
        raw = both.view(torch.uint8) if kind == "e4m3" else both
        assert not bool(raw[:, 1].float().any())
        touched = torch.zeros((cache.n_pages, 16), dtype=torch.bool, device=dev)
        for r, p in zip(req.tolist(), pos.tolist()):
            touched[int(cache.table[r, p // 16]), p % 16] = True
        assert not bool(raw[:, 0][~touched].float().any())
        assert bool((raw[:, 0][touched].float() != 0).all())
        if kind == "e4m3":
            keep = ~touched[:, None, :].expand_as(cache.k_scale)
            assert torch.equal(cache.k_scale[keep], before[0][keep])
            assert torch.equal(cache.v_scale[keep], before[1][keep])
        assert int(st) == 0


@pytest.mark.parametrize("D", [64, 34])
def test_e4m3_edges(api, dev, D):
    """Heads of zeros, of tiny and of huge values, ties, a NaN and an infinity."""
    rows = torch.zeros((8, 1, D), device=dev)
    rows[1] = 1e-42
    rows[2] = 3e38
    rows[3, 0, 0] = 448.0
    rows[3, 0, 1:5] = torch.tensor([17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10], device=dev)  # ties
    rows[4, 0, 3] = math.nan
    rows[5, 0, 2] = -math.inf
    rows[6] = -1.0
    rows[7, 0, :2] = torch.tensor([1.0, 2.0 ** -30], device=dev)
    gen = torch.Generator().manual_seed(1)
    cache = wo.Cache(gen, "e4m3", [8], 1, D, 16, filled=False)
    st = _status(dev)
    i = torch.arange(8, dtype=torch.int32, device=dev)
    api.dspark_kv_append(rows, rows, cache.kv(), req=torch.zeros_like(i), pos=i, status=st)
    assert int(st) == api.STATUS_BAD_INPUT
    out = torch.zeros((8, 1, D), device=dev)
    api.dspark_kv_read(cache.kv(), start=torch.zeros(1, dtype=torch.int32, device=dev),
                       cu_rows=torch.tensor([0, 8], dtype=torch.int32, device=dev), k_out=out,
                       v_out=torch.zeros_like(out), status=st)
    assert bool(torch.isnan(out[4]).all()) and bool(torch.isnan(out[5]).all())
    assert not bool(out[0].any()) and bool((out[1].abs() < 1e-30).all())
    assert out[3, 0, :5].tolist() == [448.0, 16.0, 20.0, 0.0, 2.0 ** -8]
    for r in (2, 6, 7):
        x = rows[r].double()
        s = x.abs().amax() / 448
        assert bool(((out[r].double() - x).abs() <= s * (wo.e4m3_step(x / s) / 2 + 1e-4)).all())


def test_append_bad_indices(api, dev):
    gen = torch.Generator().manual_seed(2)
    cache = wo.Cache(gen, "bf16", [40, 20], 1, 64, 16, filled=False)
    cache.table[1, 1] = cache.n_pages  # a page outside the pool
    req = torch.tensor([0, 0, 1, 1, 2, 0], dtype=torch.int32, device=dev)
    pos = torch.tensor([0, 48, 3, 17, 0, -5], dtype=torch.int32, device=dev)
    k = torch.ones((6, 1, 64), device=dev, dtype=torch.bfloat16)
    st = _status(dev)
    api.dspark_kv_append(k, k, cache.kv(), req=req, pos=pos, status=st)
    assert int(st) == api.STATUS_BAD_INDEX
    assert int((cache.k != 0).any(-1).sum()) == 2 and int((cache.v != 0).any(-1).sum()) == 2
    assert bool(cache.values("k", 0, 0, 1).all()) and bool(cache.values("k", 1, 3, 4).all())


def test_read_bounds(api, dev):
    gen = torch.Generator().manual_seed(4)
    cache = wo.Cache(gen, "bf16", [40, 20], 1, 64, 16)
    st = _status(dev)
    start = torch.tensor([30, -1], dtype=torch.int32, device=dev)
    cu = torch.tensor([0, 30, 32], dtype=torch.int32, device=dev)
    ko = torch.full((32, 1, 64), 9.0, device=dev)
    vo = ko.clone()
    api.dspark_kv_read(cache.kv(), start=start, cu_rows=cu, k_out=ko, v_out=vo, status=st)
    assert int(st) == api.STATUS_BAD_INDEX
    assert torch.equal(ko[:18].double(), cache.values("k", 0, 30, 48))  # 48 positions in the table
    assert bool((ko[18:31] == 9).all())
    assert torch.equal(vo[31].double(), cache.values("v", 1, 0, 1)[0])
    st.zero_()
    api.dspark_kv_read(cache.kv(), start=start.clamp(min=0), cu_rows=cu, k_out=ko, v_out=vo,
                       status=st, max_rows=7)
    assert int(st) == api.STATUS_CAPACITY


def test_offsets_past_32_bits(api, dev):
    """A pool of more than 2^32 elements: entries of its last page."""
    gen = torch.Generator().manual_seed(5)
    page, heads, D = 1024, 8, 128
    n = (1 << 32) // (page * heads * D) + 2
    k = torch.zeros((n, page, heads, D), device=dev, dtype=torch.uint8).view(torch.float8_e4m3fn)
    v = torch.zeros_like(k)
    s = [torch.zeros((n, heads, page), device=dev) for _ in range(2)]
    table = torch.tensor([[0, n - 1]], dtype=torch.int32, device=dev)
    kv = api.KVCache(k, v, table, *s)
    x = torch.randn((3, heads, D), device=dev, generator=torch.Generator("cuda").manual_seed(1)).bfloat16()
    pos = torch.tensor([page - 1, page, 2 * page - 1], dtype=torch.int32, device=dev)
    st = _status(dev)
    api.dspark_kv_append(x, -x, kv, req=torch.zeros_like(pos), pos=pos, status=st)
    out = [torch.zeros((2, heads, D), device=dev) for _ in range(2)]
    api.dspark_kv_read(kv, start=torch.tensor([2 * page - 2], dtype=torch.int32, device=dev),
                       cu_rows=torch.tensor([0, 2], dtype=torch.int32, device=dev), k_out=out[0],
                       v_out=out[1], status=st)
    assert int(st) == 0
    assert not bool(out[0][0].any())
    y = x[2].double()
    scale = y.abs().amax(-1, keepdim=True) / 448
    for o, sign in ((out[0][1], 1), (out[1][1], -1)):
        assert bool(((sign * o.double() - y).abs() <= scale * (wo.e4m3_step(y / scale) / 2 + 1e-4)).all())


def test_runs_on_the_stream_it_is_given(api, dev):
    """Inputs made on a side stream, the call enqueued there."""
    gen = torch.Generator().manual_seed(6)
    cache = wo.Cache(gen, "bf16", [300], 2, 64, 16, filled=False)
    side = torch.cuda.Stream()
    st = _status(dev)
    i = torch.arange(256, dtype=torch.int32, device=dev)
    req = torch.zeros_like(i)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        k = torch.full((256, 2, 64), 2.5, device=dev, dtype=torch.bfloat16)
        api.dspark_kv_append(k, k, cache.kv(), req=req, pos=i, status=st)
    side.synchronize()
    assert bool((cache.values("k", 0, 0, 256) == 2.5).all())


def test_argument_errors(api, dev):
    gen = torch.Generator().manual_seed(7)
    cache = wo.Cache(gen, "bf16", [16], 2, 64, 16)
    kv, st = cache.kv(), _status(dev)
    k = torch.zeros((4, 2, 64), device=dev, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32, device=dev)
    with pytest.raises(ValueError):
        api.dspark_kv_append(k[:, :1], k, kv, req=i, pos=i, status=st)  # heads
    with pytest.raises(ValueError):
        api.dspark_kv_append(k, k.float(), kv, req=i, pos=i, status=st)  # types differ
    with pytest.raises(ValueError):
        api.dspark_kv_append(k, k, kv, req=i[:3], pos=i, status=st)
    with pytest.raises(api.DsparkError):
        api.dspark_kv_append(k, k, kv, req=i, status=st)  # no positions
    with pytest.raises(api.DsparkError):
        api.dspark_kv_append(k, k, kv, req=i, pos=i, cos_sin=_angles(4, 66)[:, :66], status=st)
    with pytest.raises(ValueError):
        api.dspark_kv_append(k.transpose(0, 1), k, kv, req=i, pos=i, status=st)
    with pytest.raises(ValueError):
        api.KVCache(cache.k, cache.v[:, :8], cache.table)
    with pytest.raises(ValueError):
        api.KVCache(cache.k, cache.v, cache.table, k_scale=torch.zeros(1, device=dev))
    with pytest.raises(ValueError):
        api.KVCache(cache.k.view(torch.float16), cache.v.view(torch.float16), cache.table)
    with pytest.raises(ValueError):
        api.dspark_kv_read(kv, start=i[:1], cu_rows=i[:1], k_out=k, v_out=k, status=st)
    with pytest.raises(ValueError):
        api.dspark_qk_norm_rope(None, None, status=st)
    assert int(st) == 0


@pytest.mark.parametrize("D", [64, 128])
def test_codes_are_the_rounded_quotients(api, dev, D):
    """Every code is the 32-bit quotient x / scale rounded to nearest even, bit for
    bit, for heads of all magnitudes with large and small elements."""
    rows, heads, page = 4096, 8, 64
    g = torch.Generator("cuda").manual_seed(60)
    x = torch.randn((rows, heads, D), generator=g, device="cuda")
    x *= torch.exp2(torch.randint(-90, 90, (rows, heads, 1), generator=g, device="cuda").float())
    x *= torch.exp2(torch.randint(-12, 1, x.shape, generator=g, device="cuda").float())
    i32 = dict(dtype=torch.int32, device="cuda")
    k, v = (torch.zeros((rows // page, page, heads, D), device="cuda", dtype=torch.uint8)
            .view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.zeros((rows // page, heads, page), device="cuda") for _ in range(2))
    kv = api.KVCache(k, v, torch.arange(rows // page, **i32).view(1, -1), ks, vs)
    status = torch.zeros(1, **i32)
    api.dspark_kv_append(x, -x, kv, req=torch.zeros(rows, **i32), pos=torch.arange(rows, **i32),
                         status=status)
    torch.cuda.synchronize()
    # (by 64 bits: a quotient of 24-bit numbers rounded twice this way is the quotient
    # rounded once, while torch may divide by a number as it multiplies by its inverse)
    scale = (x.abs().amax(-1).double() / 448).float().clamp_min(2.0 ** -100)
    want = (x.double() / scale[..., None].double()).float().to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(ks.transpose(1, 2).reshape(rows, heads), scale)
    assert torch.equal(k.view(torch.uint8).view(rows, heads, D), want)
    assert torch.equal(v.view(torch.uint8).view(rows, heads, D), want ^ 0x80)
    assert int(status) == 0
