"""Guard bands around what the latent cache's and the short cache's calls write: outputs,
workspaces, ledgers and page pools are cut from the middle of larger buffers, whose borders
stay as they were."""

import pytest
import torch

import latent_oracle as lo
import window_oracle as wo
from gpu_helpers import require_gpu
from test_gpu_evict import Evicting, Gathering
from test_gpu_latent import Problem as Absorbed
from test_gpu_prompt import Problem as Prompt
from test_gpu_window_guards import Guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    require_gpu()
    from confidence_scheduled_speculative_gb300 import api
    return api


I32 = dict(dtype=torch.int32, device="cuda")


def space(g, n):
    return g.like(torch.empty(n, dtype=torch.uint8, device="cuda"), fill=0xFF)


@pytest.mark.parametrize("case", [
    dict(prefix=[100, 0, 33], win=[1, 9, 4], hq=16, page=16),
    dict(prefix=[3000, 0, 700, 65], win=[9, 0, 32, 17], hq=16, page=64),
    dict(prefix=[3000, 700], win=[30, 32], hq=64, page=64),  # teams
    dict(prefix=[90, 7], win=[3, 2], hq=3, page=7, kind="f32", dtype="f32", latent=34, rope=6),
])
def test_latent_attention_writes_its_rows_alone(api, case):
    plain = Absorbed(601, pad=0, **case).run(api)
    p = Absorbed(601, pad=0, **case)
    g = Guarded()
    p.out, p.lse = g.like(p.out), g.like(p.lse)
    before = p.cache.pool.clone()
    p.run(api, ws=space(g, api.dspark_latent_attention_workspace_bytes(p.hq, p.cache.latent)))
    g.check()
    assert torch.equal(p.out, plain.out) and torch.equal(p.lse, plain.lse)
    assert torch.equal(p.cache.pool, before) and int(p.status) == 0


@pytest.mark.parametrize("latent,rope,page,heads,kind", [(512, 64, 16, 128, "bf16"), (512, 64, 64, 20, "f32"),
                                                         (34, 6, 5, 3, "bf16")])
def test_latent_append_writes_its_rows_alone(api, latent, rope, page, heads, kind):
    gen = torch.Generator().manual_seed(602)
    c = lo.Latent(gen, kind, [60, 1, 50], page, latent, rope, filled=False)
    g = Guarded()
    c.pool = c.pages = g.like(c.pool)
    prefix, win = [50, 0, 16], [10, 1, 34]
    rows = sum(win)
    x = torch.randn((rows, latent + rope), device="cuda").bfloat16()
    q = torch.randn((rows, heads, rope), device="cuda").bfloat16()
    out = g.like(q, fill=0)
    status = torch.zeros(1, **I32)
    req = torch.repeat_interleave(torch.arange(3), torch.tensor(win)).to(**I32)
    pos = torch.cat([torch.arange(a, a + b) for a, b in zip(prefix, win)]).to(**I32)
    turn = torch.cat([torch.ones((60, rope // 2)), torch.zeros((60, rope // 2))], 1).cuda()
    api.dspark_latent_append(x, c.lc(), req=req, pos=pos, cos_sin=turn, q_rope=q, q_rope_out=out, status=status)
    g.check()
    assert torch.equal(out, q) and int(status) == 0
    got = torch.cat([c.entries(r, a, a + b) for r, (a, b) in enumerate(zip(prefix, win))])
    assert torch.equal(got, x.to(got.dtype)) and int((c.pool != 0).any(2).sum()) == rows


@pytest.mark.parametrize("case", [
    dict(lens=[(1, 1), (300, 420), (17, 17)], hq=4, hkv=2),
    dict(lens=[(513, 513)], hq=2, S=0),
    dict(lens=[(1, 1)] * 200 + [(600, 700)], hq=2),
    dict(lens=[(70, 90), (3, 3)], hq=4, hkv=2, K=33, S=7, V=50),
])
def test_prompts_write_their_rows_alone(api, case):
    plain = Prompt(603, pad=0, **case).run(api)
    p = Prompt(603, pad=0, **case)
    g = Guarded()
    p.out, p.lse = g.like(p.out), g.like(p.lse)
    p.run(api)
    g.check()
    assert torch.equal(p.out, plain.out) and torch.equal(p.lse, plain.lse) and int(p.status) == 0


@pytest.mark.parametrize("kind,dtype,D,page", [("bf16", "bf16", 128, 16), ("e4m3", "bf16", 64, 48), ("f32", "f32", 80, 7)])
@pytest.mark.parametrize("win", [[1, 1, 1], [9, 0, 32]])
def test_gathering_writes_its_ledger_alone(api, kind, dtype, D, page, win):
    case = dict(prefix=[3000, 0, 65], win=win, hq=16, hkv=2, D=D, page=page, kind=kind, dtype=dtype)
    plain = Gathering(api, 604, **case).gather(api)
    p = Gathering(api, 604, **case)
    g = Guarded()
    p.weights, p.positions = g.like(p.weights), g.like(p.positions)
    before = [t.view(torch.uint8).clone() for t in (p.cache.k, p.cache.v)]
    p.gather(api)
    g.check()
    assert torch.equal(p.weights, plain.weights) and torch.equal(p.positions, plain.positions)
    assert all(torch.equal(a, b.view(torch.uint8)) for a, b in zip(before, (p.cache.k, p.cache.v)))
    assert int(p.status) == 0


@pytest.mark.parametrize("case", [
    dict(lens=[300, 20, 299], keep=20, recent=0, kind="e4m3", D=128, page=64),
    dict(lens=[10000, 70], keep=4096, recent=64, hkv=1, page=64),
    dict(lens=[20000, 17, 16385], keep=9000, recent=50, D=64, page=64),
    dict(lens=[400000, 393217], keep=200000, recent=100, hkv=1, D=16, page=256),
    dict(lens=[90, 33], keep=31, recent=3, D=34, page=7, kind="f32"),
])
def test_eviction_writes_its_cache_and_ledger_alone(api, case):
    plain = Evicting(605, **case).run(api, inplace=True)
    e = Evicting(605, **case)
    g, c = Guarded(), e.cache
    c.k, c.v = (g.like(t.view(torch.uint8)).view(t.dtype) for t in (c.k, c.v))
    if c.k_scale is not None:
        c.k_scale, c.v_scale = g.like(c.k_scale), g.like(c.v_scale)
    w, p, lens = g.like(e.weights), g.like(e.positions), g.like(e.n)
    ws = space(g, api.dspark_kv_evict_workspace_bytes(len(e.lens), e.hkv, e.length))
    api.dspark_kv_evict(c.kv(), lens=lens, now=e.now, keep=e.keep, recent=e.recent, weights=w, positions=p,
                        workspace=ws, status=e.status)
    g.check()
    assert torch.equal(w, plain.w) and torch.equal(p, plain.p) and torch.equal(lens, plain.new)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8))
               for a, b in ((c.k, plain.cache.k), (c.v, plain.cache.v)))
    assert int(e.status) == 0
