"""Heads that are not a power of two of eight elements: the lanes of a warp beyond a head
take no part in its norm, its largest element or its scale."""

import pytest
import torch

import window_oracle as wo
from gpu_helpers import require_gpu
from test_gpu_cache import _angles, _check_stored, _close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    require_gpu()
    from confidence_scheduled_speculative_gb300 import api
    return api


@pytest.mark.parametrize("D", [8, 16, 24, 40, 48, 56, 72, 80, 96, 112, 136, 192, 248])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv", [(0, 8), (10, 5), (2, 2), (24, 3)])
def test_every_scale_is_the_heads_own(api, D, dtype, hq, hkv):
    """Norm weights with and without rotation, hundreds of rows, into E4M3."""
    gen, g = torch.Generator().manual_seed(D), torch.Generator("cuda").manual_seed(D + hq)
    dt, rows = wo.DTYPES[dtype], 400
    i32 = dict(dtype=torch.int32, device="cuda")
    x = (torch.randn((rows, hq + 2 * hkv, D), generator=g, device="cuda") * 2).to(dt)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    weight = (1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(dt)
    pos = torch.arange(rows, **i32)
    for rope in (0, 8, D):
        cache = wo.Cache(gen, "e4m3", [rows], hkv, D, 16, filled=False)
        table = _angles(rows, rope) if rope else None
        status, q_out = torch.zeros(1, **i32), torch.zeros((rows, hq, D), device="cuda", dtype=dt)
        api.dspark_kv_append(k, v, cache.kv(), q=q if hq else None, q_out=q_out if hq else None,
                             req=torch.zeros(rows, **i32), pos=pos, q_weight=weight, k_weight=weight,
                             cos_sin=table, status=status)
        assert int(status) == 0
        y, tol = wo.norm_rope(k, weight, 1e-6, table, pos, False)
        _check_stored(cache, "k", 0, (0, rows), y, tol)
        _check_stored(cache, "v", 0, (0, rows), v.double(), torch.zeros_like(v, dtype=torch.float64))
        if hq:
            y, tol = wo.norm_rope(q, weight, 1e-6, table, pos, False)
            _close(q_out, y, tol, wo.out_unit(dt))
