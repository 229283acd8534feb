"""Calls of the attention side of a window that have to be refused or flagged, each
beside what has to go on working."""

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


# A bfloat16 cache and an E4M3 one on the tensor cores (the latter with eight query rows
# a step and, nine heads a key head, with 64), and 32 bits.
KINDS = [("bf16", "bf16", 2, 64), ("e4m3", "bf16", 4, 64), ("e4m3", "bf16", 9, 128), ("f32", "f32", 2, 64)]


@pytest.mark.parametrize("kind,dtype,group,D", KINDS)
@pytest.mark.parametrize("first", [2 ** 31 - 5, 2 ** 31 - 8195])
def test_positions_that_32_bits_cannot_count(api, kind, dtype, group, D, first):
    """A table that lists 2^31 positions: the last of them are more than the kernels'
    counters hold.  The request is flagged, the others come out right."""
    page = 1 << 16
    p = Problem(500, [40, 100, 700], [4, 4, 3], group, 1, D, page, kind, dtype=dtype)
    table = torch.zeros((3, (1 << 31) // page), dtype=torch.int32, device="cuda")
    table[:, :p.cache.table.size(1)] = p.cache.table
    p.cache.table = table
    p.prefix_lens[1] = first
    p.run(api).check(skip=(1,))
    assert int(p.status) == api.STATUS_BAD_INDEX


def test_output_beside_the_queries(api):
    """Queries and outputs as slices of one buffer: side by side, after one another, and
    in rows of different strides.  Over one another they are refused, and nothing is
    written."""
    for kind, dtype, group, D in KINDS:
        p = Problem(510, [600, 30], [9, 5], group, 1, D, 64, kind, dtype=dtype, pad=0)
        n = p.rows
        both = torch.zeros((2 * n, 2 * group, D), device="cuda", dtype=p.dtype)
        for q, out in ((both[:n, :group], both[:n, group:]), (both[n:, group:], both[:n, group:]),
                       (both[:n, group:], both.view(4 * n, group, D)[2 * n:3 * n])):
            q.copy_(p.q)
            p.q, p.out = q, out
            p.run(api).check()
            assert int(p.status) == 0
        before = both.clone()
        for q, out in ((both[:n, :group], both[:n, :group]), (both[:n, :group], both[1:n + 1, :group]),
                       (both[:n, :group], both.view(4 * n, group, D)[:n])):
            p.q, p.out = q, out
            with pytest.raises(api.DsparkError):
                p.run(api)
        assert torch.equal(before, both)


@pytest.mark.parametrize("kind,dtype,group,D", KINDS)
def test_windows_outside_the_rows(api, kind, dtype, group, D):
    """A window that begins behind the last row, or ends before it begins, is flagged in
    every kernel, not left out without a word."""
    def call(p, rows):
        ws = api.workspace(api.dspark_tree_attention_workspace_bytes(p.hq, p.D))
        api.dspark_tree_attention(p.q, p.cache.kv(), cu_seqlens=p.cu, prefix_lens=p.prefix_lens,
                                  scale=p.scale, out=p.out, lse=p.lse, workspace=ws, status=p.status,
                                  max_rows=rows)
        torch.cuda.synchronize()

    p = Problem(520, [40, 20, 33], [4, 3, 2], group, 1, D, 64, kind, dtype=dtype)
    call(p, 7)  # the third request's rows are 7 and 8
    p.rows = 7
    p.check(skip=(2,))
    assert int(p.status) == api.STATUS_BAD_LEN
    p = Problem(521, [40, 20, 33], [4, 3, 0], group, 1, D, 64, kind, dtype=dtype)
    p.cu[3] = 5  # the third request: rows 7 to 5
    call(p, 7)
    assert int(p.status) == api.STATUS_BAD_LEN


@pytest.mark.parametrize("kind,dtype,D", [("bf16", "bf16", 64), ("e4m3", "bf16", 128), ("f32", "f32", 34)])
def test_a_row_that_cannot_be_rotated_is_not_stored(api, kind, dtype, D):
    """A position outside the rotation's table: neither the row's key nor its value (nor
    its query) is written, so that the slot keeps what it held as a whole."""
    gen = torch.Generator().manual_seed(530)
    c = wo.Cache(gen, kind, [40], 2, D, 16)
    x = torch.randn((4, 6, D), device="cuda").to(wo.DTYPES[dtype])
    i32 = dict(dtype=torch.int32, device="cuda")
    cos_sin = torch.zeros((10, 2), device="cuda")
    before = {n: c.values(n, 0, 0, 40) for n in "kv"}
    q_out, status = torch.full((4, 2, D), 7.0, device="cuda", dtype=x.dtype), torch.zeros(1, **i32)
    api.dspark_kv_append(x[:, 2:4], x[:, 4:], c.kv(), q=x[:, :2], q_out=q_out, req=torch.zeros(4, **i32),
                         pos=torch.tensor([9, 10, -1, 0], **i32), cache_pos=torch.tensor([5, 6, 7, 39], **i32),
                         cos_sin=cos_sin, status=status)
    assert int(status) == api.STATUS_BAD_INDEX
    assert bool((q_out[1:3] == 7).all()) and bool((q_out[[0, 3]] != 7).all())
    for n, t in before.items():
        same = (c.values(n, 0, 0, 40) == t).flatten(1).all(1)
        assert same.nonzero()[:, 0].tolist() == [p for p in range(40) if p not in (5, 39)], n


def test_windows_without_rows(api):
    """A step in which no row is left: every call takes tensors of no rows and does
    nothing."""
    c = wo.Cache(torch.Generator().manual_seed(540), "bf16", [40, 3], 2, 64, 16)
    i32 = dict(dtype=torch.int32, device="cuda")
    x = torch.zeros((0, 8, 64), device="cuda", dtype=torch.bfloat16)
    none, status = torch.zeros(0, **i32), torch.zeros(1, **i32)
    before = [t.clone() for t in (c.k, c.v)]
    api.dspark_qk_norm_rope(x[:, :4], x[:, 4:6], pos=none, cos_sin=torch.ones((9, 64), device="cuda"),
                            status=status)
    api.dspark_kv_append(x[:, 4:6], x[:, 6:], c.kv(), q=x[:, :4], req=none, pos=none, status=status)
    zeros = torch.zeros(3, **i32)
    api.dspark_kv_read(c.kv(), start=zeros[:2], cu_rows=zeros, k_out=x[:, :2], v_out=x[:, 2:4],
                       status=status)
    ws = api.workspace(api.dspark_tree_attention_workspace_bytes(4, 64))
    api.dspark_tree_attention(x[:, :4], c.kv(), cu_seqlens=zeros, prefix_lens=zeros[:2], scale=0.125,
                              out=x[:, 4:], ancestors=none, lse=torch.zeros((0, 4), device="cuda"),
                              workspace=ws, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0 and all(torch.equal(a, b) for a, b in zip(before, (c.k, c.v)))


def test_outputs_without_their_inputs(api):
    """An output whose input is not given would stay unwritten: refused."""
    c = wo.Cache(torch.Generator().manual_seed(550), "bf16", [40], 2, 64, 16)
    x = torch.zeros((3, 8, 64), device="cuda", dtype=torch.bfloat16)
    i, status = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="q_out"):
        api.dspark_kv_append(x[:, :2], x[:, 2:4], c.kv(), req=i, pos=i, q_out=x[:, 4:], status=status)
    with pytest.raises(ValueError, match="k_out"):
        api.dspark_qk_norm_rope(x[:, :2], None, k_out=x[:, 4:], status=status)
    with pytest.raises(ValueError, match="q_out"):
        api.dspark_qk_norm_rope(None, x[:, :2], q_out=x[:, 4:], status=status)
