"""Host-side argument checks of the verify window's cache operators: each
rejected call returns its code before anything is enqueued (no GPU)."""

import ctypes

import pytest

from test_abi import FAKE, lib  # noqa: F401 (a fixture)


def _api():
    from confidence_scheduled_speculative_gb300 import api
    return api


def _cache(**over):
    f = FAKE.value
    fields = dict(dtype=0, n_pages=4, page_size=16, n_kv_heads=2, head_dim=64, n_requests=3,
                  table_width=2, page_stride=2048, token_stride=128, head_stride=64, k=f, v=f,
                  k_scale=None, v_scale=None, block_table=f)
    return _api().dspark_kv_cache(**{**fields, **over})


BAD_CACHES = [dict(dtype=3), dict(dtype=2), dict(dtype=2, k_scale=FAKE.value), dict(n_pages=0),
              dict(page_size=0), dict(n_kv_heads=0), dict(n_requests=0), dict(table_width=0),
              dict(page_stride=-1), dict(token_stride=-1), dict(head_stride=-1), dict(k=None),
              dict(v=None), dict(block_table=None)]


def _i64(x):
    return ctypes.c_int64(x)


def _norm_rope(lib, nr=None, q=FAKE, ld_q=256, k=FAKE, ld_k=128, dtype=0, hq=4, hkv=2, D=64,
               pos=FAKE, rows=8, qo=FAKE, lqo=256, ko=FAKE, lko=128, status=FAKE, **over):
    fields = dict(q_weight=None, k_weight=None, eps=1e-6, cos_sin=FAKE.value, n_pos=10, rope_dim=64,
                  interleaved=0)
    nr = _api().dspark_norm_rope(**{**fields, **over}) if nr is None else nr
    f = lib.dspark_qk_norm_rope
    f.restype = ctypes.c_int
    return f(q, _i64(ld_q), k, _i64(ld_k), dtype, hq, hkv, D, ctypes.byref(nr) if nr else None, pos,
             None, rows, qo, _i64(lqo), ko, _i64(lko), status, None)


def test_norm_rope_checks(lib):  # noqa: F811
    assert _norm_rope(lib, rows=0) == 0  # nothing to do
    assert _norm_rope(lib, nr=False) == -1
    for bad in (dict(q=None), dict(qo=None), dict(k=None), dict(ko=None), dict(ld_q=255),
                dict(ld_k=127), dict(lqo=255), dict(lko=127), dict(dtype=2), dict(hq=0),
                dict(hkv=0), dict(hq=-1), dict(rows=-1), dict(status=None), dict(pos=None),
                dict(rope_dim=63), dict(rope_dim=0), dict(rope_dim=66), dict(n_pos=-1),
                dict(eps=-1.0), dict(eps=float("nan"))):
        assert _norm_rope(lib, **bad) == -1, bad
    assert _norm_rope(lib, q=None, qo=None, hq=0, k=None, ko=None, hkv=0) == -1
    assert _norm_rope(lib, D=258, ld_q=2000, ld_k=2000, lqo=2000, lko=2000) == -4
    assert _norm_rope(lib, D=63) == -4


def _append(lib, cache, k=FAKE, v=FAKE, ld_v=128, req=FAKE, pos=FAKE, cache_pos=None, q=FAKE,
            qo=FAKE, hq=4, dtype=0, rows=0, status=FAKE):
    f = lib.dspark_kv_append
    f.restype = ctypes.c_int
    return f(q, _i64(256), k, _i64(128), v, _i64(ld_v), dtype, hq,
             None if cache is None else ctypes.byref(cache), None, req, pos, cache_pos, None, rows,
             qo, _i64(256), status, None)


def test_append_checks(lib):  # noqa: F811
    assert _append(lib, _cache()) == 0
    assert _append(lib, _cache(dtype=2, k_scale=FAKE.value, v_scale=FAKE.value)) == 0
    assert _append(lib, _cache(), pos=None, cache_pos=FAKE) == 0
    assert _append(lib, _cache(), q=None, qo=None, hq=0) == 0
    assert _append(lib, None) == -1
    for bad in BAD_CACHES:
        assert _append(lib, _cache(**bad)) == -1, bad
    for bad in (dict(k=None), dict(v=None), dict(req=None), dict(pos=None), dict(ld_v=127),
                dict(q=None), dict(qo=None), dict(hq=0), dict(dtype=2), dict(rows=-1),
                dict(status=None)):
        assert _append(lib, _cache(), **bad) == -1, bad
    assert _append(lib, _cache(head_dim=258)) == -4
    assert _append(lib, _cache(head_dim=7)) == -4


def _read(lib, cache, start=FAKE, cu=FAKE, B=3, rows=0, dtype=0, ko=FAKE, vo=FAKE, ld=128, st=FAKE):
    f = lib.dspark_kv_read
    f.restype = ctypes.c_int
    return f(None if cache is None else ctypes.byref(cache), start, cu, B, rows, dtype, ko, vo,
             _i64(ld), st, None)


def test_read_checks(lib):  # noqa: F811
    assert _read(lib, _cache()) == 0
    assert _read(lib, None) == -1
    for bad in BAD_CACHES:
        assert _read(lib, _cache(**bad)) == -1, bad
    for bad in (dict(start=None), dict(cu=None), dict(B=0), dict(B=4), dict(rows=-1), dict(dtype=2),
                dict(ko=None), dict(vo=None), dict(ld=127), dict(st=None)):
        assert _read(lib, _cache(), **bad) == -1, bad
    assert _read(lib, _cache(head_dim=300), ld=1000) == -4


def _attend(lib, cache, q=FAKE, ld_q=256, dtype=0, hq=4, rows=0, cu=FAKE, prefix=FAKE, B=3,
            scale=0.125, out=FAKE, ld_out=256, ws=FAKE, ws_bytes=None, st=FAKE):
    f = lib.dspark_tree_attention
    f.restype = ctypes.c_int
    need = lib.dspark_tree_attention_workspace_bytes
    need.restype = ctypes.c_size_t
    n = need(4, 64) if ws_bytes is None else ws_bytes
    return f(q, _i64(ld_q), dtype, hq, rows, cu, prefix, B, None, ctypes.c_float(scale),
             None if cache is None else ctypes.byref(cache), out, _i64(ld_out), None, ws,
             ctypes.c_size_t(n), st, None)


def test_attention_checks(lib):  # noqa: F811
    assert _attend(lib, _cache()) == 0
    assert _attend(lib, None) == -1
    for bad in BAD_CACHES:
        assert _attend(lib, _cache(**bad)) == -1, bad
    for bad in (dict(q=None), dict(out=None), dict(cu=None), dict(prefix=None), dict(st=None),
                dict(ld_q=255), dict(ld_out=255), dict(dtype=2), dict(hq=3), dict(hq=0),
                dict(rows=-1), dict(B=0), dict(B=4), dict(scale=float("nan")),
                dict(scale=float("inf"))):
        assert _attend(lib, _cache(), **bad) == -1, bad
    assert _attend(lib, _cache(head_dim=7)) == -4
    assert _attend(lib, _cache(), ws=None) == -2
    assert _attend(lib, _cache(), ws=ctypes.c_void_p(0x10010)) == -2
    assert _attend(lib, _cache(), ws_bytes=8) == -2


@pytest.mark.parametrize("hq,D,ok", [(1, 2, True), (64, 128, True), (0, 64, False), (4, 0, False),
                                     (4, 258, False)])
def test_attention_workspace(lib, hq, D, ok):  # noqa: F811
    f = lib.dspark_tree_attention_workspace_bytes
    f.restype = ctypes.c_size_t
    assert (f(hq, D) > 0) == ok and f(hq, D) % 256 == 0
