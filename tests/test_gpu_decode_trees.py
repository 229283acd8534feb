"""PagedCache over trees of drafted tokens: what a branch gets is what the same tokens
get as a chain of their own."""

import pytest
import torch

import window_oracle as wo
from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def decode():
    require_gpu()
    from confidence_scheduled_speculative_gb300 import decode
    return decode


def _angles(n, D):
    a = torch.arange(n, device="cuda").double()[:, None] * 10000.0 ** (
        -torch.arange(0, D, 2, device="cuda").double() / D)
    return torch.cat([a.cos(), a.sin()], 1).float()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_a_tree_of_branches(decode, kind):
    """A prefix, then a tree of two branches that share their first token, against the
    definition in 64 bits of either branch as a chain after the prefix."""
    hq, hkv, D, P = 4, 2, 64, 37
    dt = wo.DTYPES[kind]
    gen = torch.Generator("cuda").manual_seed(7)
    i32 = dict(dtype=torch.int32, device="cuda")
    status = torch.zeros(1, **i32)
    cache = decode.PagedCache(1, 64, hq, hkv, D, page_size=16, dtype=dt, seed=3)
    table = _angles(64, D)
    parent = [-1, 0, 0, 1, 2, 3, 4, 4]  # of each token of the window
    L = len(parent)
    depth, bits = [], []
    for i, p in enumerate(parent):
        depth.append(depth[p] + 1 if p >= 0 else 0)
        bits.append((bits[p] if p >= 0 else 0) | 1 << i)
    x = torch.randn((P + L, hq + 2 * hkv, D), generator=gen, device="cuda").to(dt)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    rotated = torch.empty((P + L, hq, D), device="cuda", dtype=dt)
    pos = torch.tensor(list(range(P)) + [P + d for d in depth], **i32)
    place = torch.arange(P + L, **i32)
    for lo, hi in ((0, P), (P, P + L)):
        cache.append(q[lo:hi], k[lo:hi], v[lo:hi], req=torch.zeros(hi - lo, **i32), pos=pos[lo:hi],
                     cache_pos=place[lo:hi], q_out=rotated[lo:hi], cos_sin=table, status=status)
    out = torch.zeros((L, hq, D), device="cuda", dtype=dt)
    cache.attend(rotated[P:], out, cu_seqlens=torch.tensor([0, L], **i32),
                 prefix_lens=torch.tensor([P], **i32), scale=D ** -0.5, status=status,
                 ancestors=wo.as_int32(bits).cuda())
    torch.cuda.synchronize()
    assert int(status) == 0
    unit = wo.out_unit(dt)
    y, tol = wo.norm_rope(torch.cat([q, k], 1), None, 0.0, table, pos, False)
    for i in range(L):
        path = list(range(P)) + [P + j for j in range(L) if bits[i] >> j & 1]
        kk = y[path][:, hq:].repeat_interleave(hq // hkv, 1)
        vv = v[path].double().repeat_interleave(hq // hkv, 1)
        qq = y[P + i, :hq]
        s = torch.einsum("hd,nhd->hn", qq, kk) * D ** -0.5
        w = s.softmax(-1)
        want, size = torch.einsum("hn,nhd->hd", w, vv), torch.einsum("hn,nhd->hd", w, vv.abs())
        # queries and keys are rounded once each, a score by twice that unit of its
        # products' sizes; a weight by twice a score's error, and once to the products'
        # type; the output once; sums of D and n terms in 32 bits
        s_abs = (torch.einsum("hd,nhd->hn", qq.abs(), kk.abs()) * D ** -0.5).amax(-1, keepdim=True)
        s_tol = s_abs * (2 * unit + (2 * D + 16) * wo.U32)
        bound = size * (2 * s_tol + unit + (2 * len(path) + 32) * wo.U32) * (1 + 4 * s_tol) + unit * want.abs()
        assert bool(((out[i].double() - want).abs() <= bound).all()), i
        # and it is no chain: without the shared parent's other branch the row differs
        if 0 < i < L - 1:
            other = list(range(P)) + [P + j for j in range(i + 1)]
            if other != path:
                s2 = torch.einsum("hd,nhd->hn", qq, y[other][:, hq:].repeat_interleave(hq // hkv, 1)) * D ** -0.5
                o2 = torch.einsum("hn,nhd->hd", s2.softmax(-1),
                                  v[other].double().repeat_interleave(hq // hkv, 1))
                assert bool(((out[i].double() - o2).abs() > bound).any()), i
