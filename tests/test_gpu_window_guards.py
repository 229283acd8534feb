"""Guard bands around what the attention side of a window writes: outputs,
workspace and page pool are cut from the middle of larger buffers, whose
borders stay as they were."""

import pytest
import torch

import window_oracle as wo
from gpu_helpers import require_gpu
from test_gpu_attention import Problem

pytestmark = pytest.mark.gpu
BAND = 4096  # bytes on either side


@pytest.fixture(scope="module")
def api():
    require_gpu()
    from confidence_scheduled_speculative_gb300 import api
    return api


class Guarded:
    """Tensors inside sentinel bytes."""

    def __init__(self):
        self.kept = []

    def like(self, t, fill=None):
        n = t.numel() * t.element_size()
        raw = torch.full((n + 2 * BAND,), 0xA5, dtype=torch.uint8, device="cuda")
        inner = raw[BAND:BAND + n].view(t.dtype).view(t.shape)
        if fill is None:
            inner.view(torch.uint8).copy_(t.contiguous().view(torch.uint8))
        else:
            inner.fill_(fill)
        self.kept.append((raw, n))
        return inner

    def check(self):
        torch.cuda.synchronize()
        for raw, n in self.kept:
            assert bool((raw[:BAND] == 0xA5).all()) and bool((raw[BAND + n:] == 0xA5).all())


@pytest.mark.parametrize("kind,dtype,D,page", [("bf16", "bf16", 128, 16), ("bf16", "bf16", 64, 64),
                                               ("e4m3", "bf16", 128, 64), ("e4m3", "bf16", 64, 48),
                                               ("f32", "f32", 80, 7)])
@pytest.mark.parametrize("win", [[1, 1, 1, 1], [9, 0, 32, 17], [32, 32, 32, 32]])
def test_attention_writes_its_rows_alone(api, kind, dtype, D, page, win):
    prefix = [3000, 0, 700, 65]
    p = Problem(401, prefix, win, 8, 2, D, page, kind, dtype=dtype, pad=0)
    plain = Problem(401, prefix, win, 8, 2, D, page, kind, dtype=dtype, pad=0).run(api)
    g = Guarded()
    p.out, p.lse = g.like(p.out), g.like(p.lse)
    ws = g.like(torch.empty(api.dspark_tree_attention_workspace_bytes(8, D), dtype=torch.uint8,
                            device="cuda"), fill=0xFF)
    c = p.cache
    before = [t.clone() for t in (c.k.view(torch.uint8), c.v.view(torch.uint8))]
    api.dspark_tree_attention(p.q, c.kv(), cu_seqlens=p.cu, prefix_lens=p.prefix_lens,
                              scale=p.scale, out=p.out, lse=p.lse, workspace=ws, status=p.status)
    g.check()
    assert torch.equal(p.out, plain.out) and torch.equal(p.lse, plain.lse)
    assert all(torch.equal(a, b.view(torch.uint8)) for a, b in zip(before, (c.k, c.v)))
    assert int(p.status) == 0


@pytest.mark.parametrize("kind,dtype,D,page", [("bf16", "bf16", 128, 16), ("e4m3", "bf16", 128, 64),
                                               ("e4m3", "f32", 80, 7), ("f32", "f32", 64, 5)])
def test_append_and_read_write_their_rows_alone(api, kind, dtype, D, page):
    gen = torch.Generator().manual_seed(402)
    prefix, win = [50, 0, 16], [9, 1, 32]
    c = wo.Cache(gen, kind, [a + b for a, b in zip(prefix, win)], 2, D, page, filled=False)
    g = Guarded()
    c.k, c.v = g.like(c.k.view(torch.uint8) if kind == "e4m3" else c.k), \
        g.like(c.v.view(torch.uint8) if kind == "e4m3" else c.v)
    if kind == "e4m3":
        c.k, c.v = c.k.view(torch.float8_e4m3fn), c.v.view(torch.float8_e4m3fn)
        c.k_scale, c.v_scale = g.like(c.k_scale), g.like(c.v_scale)
    kv = c.kv()
    rows = sum(win)
    x = torch.randn((rows, 8, D), device="cuda").to(wo.DTYPES[dtype])
    q_out = g.like(x[:, :4].contiguous(), fill=0)
    i32 = dict(dtype=torch.int32, device="cuda")
    req = torch.repeat_interleave(torch.arange(3), torch.tensor(win)).to(**i32)
    pos = torch.cat([torch.arange(a, a + b) for a, b in zip(prefix, win)]).to(**i32)
    status = torch.zeros(1, **i32)
    api.dspark_kv_append(x[:, 4:6], x[:, 6:8], kv, req=req, pos=pos, q=x[:, :4], q_out=q_out,
                         status=status)
    out = [g.like(torch.empty((rows, 2, D), device="cuda"), fill=0) for _ in range(2)]
    cu = torch.tensor([0, 9, 10, 42], **i32)
    api.dspark_kv_read(kv, start=torch.tensor(prefix, **i32), cu_rows=cu, k_out=out[0],
                       v_out=out[1], status=status)
    g.check()
    assert int(status) == 0 and torch.equal(q_out, x[:, :4])
    for got, want in zip(out, (x[:, 4:6].float(), x[:, 6:8].float())):
        # E4M3: half a step of a code, 2^-4 of it, and no less than of the smallest one
        tol = want.abs() / 16 + want.abs().amax(-1, keepdim=True) * 2.0 ** -18 if kind == "e4m3" \
            else torch.zeros_like(want)
        if kind == "bf16" and dtype == "f32":
            tol = want.abs() * 2.0 ** -8
        assert bool(((got - want).abs() <= tol).all())
