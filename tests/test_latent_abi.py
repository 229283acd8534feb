"""Host-side argument checks of the latent cache's and the short cache's operators: each
rejected call returns its code before anything is enqueued (no GPU)."""

import ctypes

import pytest

from test_abi import FAKE, lib  # noqa: F401 (a fixture)
from test_window_abi import BAD_CACHES, _cache


def _api():
    from confidence_scheduled_speculative_gb300 import api
    return api


def _i64(x):
    return ctypes.c_int64(x)


def _latent(**over):
    f = FAKE.value
    fields = dict(dtype=0, n_pages=4, page_size=16, latent_dim=512, rope_dim=64, n_requests=3, table_width=2,
                  page_stride=9216, token_stride=576, data=f, block_table=f)
    return _api().dspark_latent_cache(**{**fields, **over})


BAD_LATENT = [dict(dtype=2), dict(dtype=-1), dict(n_pages=0), dict(page_size=0), dict(n_requests=0),
              dict(table_width=0), dict(page_stride=-1), dict(token_stride=-1), dict(data=None),
              dict(block_table=None)]
ODD_LATENT = [dict(latent_dim=0), dict(latent_dim=511), dict(latent_dim=514), dict(rope_dim=0), dict(rope_dim=63),
              dict(rope_dim=130)]


def _append(lib, cache, x=FAKE, ld_x=576, q=FAKE, ld_q=768, hs=192, dtype=0, hq=4, req=FAKE, pos=FAKE, rows=0,
            qo=FAKE, lqo=2304, hso=576, status=FAKE, nr=True, **over):
    fields = dict(q_weight=None, k_weight=FAKE.value, eps=1e-6, cos_sin=FAKE.value, n_pos=10, rope_dim=64,
                  interleaved=0)
    nr = _api().dspark_norm_rope(**{**fields, **over}) if nr else None
    f = lib.dspark_latent_append
    f.restype = ctypes.c_int
    return f(x, _i64(ld_x), q, _i64(ld_q), _i64(hs), dtype, hq, None if cache is None else ctypes.byref(cache),
             ctypes.byref(nr) if nr else None, req, pos, None, None, rows, qo, _i64(lqo), _i64(hso), status, None)


def test_append_checks(lib):  # noqa: F811
    assert _append(lib, _latent()) == 0
    assert _append(lib, _latent(), k_weight=None) == 0
    assert _append(lib, _latent(), q=None, qo=None, hq=0) == 0
    assert _append(lib, None) == -1
    for bad in BAD_LATENT:
        assert _append(lib, _latent(**bad)) == -1, bad
    for bad in ODD_LATENT:
        assert _append(lib, _latent(**bad)) == -4, bad
    for bad in (dict(x=None), dict(nr=False), dict(cos_sin=None), dict(q_weight=FAKE.value), dict(req=None),
                dict(pos=None), dict(status=None), dict(rows=-1), dict(hq=-1), dict(hq=0), dict(q=None),
                dict(qo=None), dict(dtype=2), dict(eps=-1.0), dict(eps=float("nan")), dict(rope_dim=32),
                dict(n_pos=-1), dict(ld_x=575), dict(hs=63), dict(hso=63), dict(ld_q=639), dict(lqo=1791)):
        assert _append(lib, _latent(), **bad) == -1, bad


def _attend(lib, cache, q=FAKE, ld_q=2304, dtype=0, hq=4, rows=0, cu=FAKE, prefix=FAKE, B=3, scale=0.04, out=FAKE,
            ld_out=2048, ws=FAKE, ws_bytes=None, st=FAKE):
    f = lib.dspark_latent_attention
    f.restype = ctypes.c_int
    need = lib.dspark_latent_attention_workspace_bytes
    need.restype = ctypes.c_size_t
    n = need(4, 512) if ws_bytes is None else ws_bytes
    return f(q, _i64(ld_q), dtype, hq, rows, cu, prefix, B, None, ctypes.c_float(scale),
             None if cache is None else ctypes.byref(cache), out, _i64(ld_out), None, ws, ctypes.c_size_t(n), st, None)


def test_attention_checks(lib):  # noqa: F811
    assert _attend(lib, _latent()) == 0
    assert _attend(lib, None) == -1
    for bad in BAD_LATENT:
        assert _attend(lib, _latent(**bad)) == -1, bad
    for bad in ODD_LATENT:
        assert _attend(lib, _latent(**bad)) == -4, bad
    for bad in (dict(q=None), dict(out=None), dict(cu=None), dict(prefix=None), dict(st=None), dict(ld_q=2303),
                dict(ld_out=2047), dict(dtype=2), dict(hq=0), dict(rows=-1), dict(B=0), dict(B=4),
                dict(scale=float("nan")), dict(scale=float("inf"))):
        assert _attend(lib, _latent(), **bad) == -1, bad
    assert _attend(lib, _latent(), hq=65536, ld_q=65536 * 576, ld_out=65536 * 512) == -4
    assert _attend(lib, _latent(), ws=None) == -2
    assert _attend(lib, _latent(), ws=ctypes.c_void_p(0x10010)) == -2
    assert _attend(lib, _latent(), ws_bytes=8) == -2
    # the output over the queries (rows that share an element)
    q, out = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x100000 + 4 * 576 * 2 - 2)
    assert _attend(lib, _latent(), q=q, out=out, rows=1) == -1


@pytest.mark.parametrize("hq,D,ok", [(1, 2, True), (128, 512, True), (0, 512, False), (4, 0, False), (4, 514, False)])
def test_attention_workspace(lib, hq, D, ok):  # noqa: F811
    f = lib.dspark_latent_attention_workspace_bytes
    f.restype = ctypes.c_size_t
    assert (f(hq, D) > 0) == ok and f(hq, D) % 256 == 0


def _prompt(lib, q=FAKE, ld_q=768, k=FAKE, ld_k=1024, hs_k=256, s=FAKE, ld_s=64, v=FAKE, ld_v=1024, hs_v=256,
            dtype=0, hq=4, hkv=4, K=128, S=64, V=128, rows=0, keys=9, cu=FAKE, cu_k=FAKE, B=3, scale=0.1, out=FAKE,
            ld_out=512, st=FAKE):
    f = lib.dspark_prompt_attention
    f.restype = ctypes.c_int
    return f(q, _i64(ld_q), k, _i64(ld_k), _i64(hs_k), s, _i64(ld_s), v, _i64(ld_v), _i64(hs_v), dtype, hq, hkv, K,
             S, V, rows, keys, cu, cu_k, B, ctypes.c_float(scale), out, _i64(ld_out), None, st, None)


def test_prompt_checks(lib):  # noqa: F811
    assert _prompt(lib) == 0
    assert _prompt(lib, s=None, S=0) == 0
    assert _prompt(lib, hkv=2) == 0
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(cu=None), dict(cu_k=None),
                dict(st=None), dict(rows=-1), dict(keys=-1), dict(B=0), dict(hq=0), dict(hkv=0), dict(hkv=3),
                dict(dtype=2), dict(s=None), dict(S=0), dict(ld_q=767), dict(ld_out=511), dict(hs_k=127),
                dict(hs_v=127), dict(ld_k=895), dict(ld_v=895), dict(ld_s=63), dict(scale=float("nan"))):
        assert _prompt(lib, **bad) == -1, bad
    for bad in (dict(K=0), dict(K=257), dict(V=0), dict(V=257), dict(S=257), dict(S=-1), dict(hq=65536, hkv=1)):
        assert _prompt(lib, **{**dict(ld_q=1 << 40, ld_out=1 << 40), **bad}) == -4, bad


def _weights(lib, cache, q=FAKE, ld_q=256, dtype=0, hq=4, rows=0, cu=FAKE, prefix=FAKE, B=3, scale=0.1, lse=FAKE,
             decay=1.0, w=FAKE, wo=FAKE, length=8, pos=None, positions=None, st=FAKE):
    f = lib.dspark_attention_weights
    f.restype = ctypes.c_int
    return f(q, _i64(ld_q), dtype, hq, rows, cu, prefix, B, None, ctypes.c_float(scale),
             None if cache is None else ctypes.byref(cache), lse, None, ctypes.c_float(decay), w, wo, length, pos,
             positions, st, None)


def test_weights_checks(lib):  # noqa: F811
    assert _weights(lib, None) == -1
    for bad in BAD_CACHES:
        assert _weights(lib, _cache(**bad)) == -1, bad
    for bad in (dict(q=None), dict(lse=None), dict(w=None), dict(wo=None), dict(cu=None), dict(prefix=None),
                dict(st=None), dict(ld_q=255), dict(dtype=2), dict(hq=3), dict(hq=0), dict(rows=-1), dict(B=0),
                dict(B=4), dict(length=0), dict(scale=float("inf")), dict(decay=float("nan")), dict(pos=FAKE),
                dict(positions=FAKE), dict(wo=ctypes.c_void_p(FAKE.value + 4))):
        assert _weights(lib, _cache(), **bad) == -1, bad
    assert _weights(lib, _cache(head_dim=258)) == -4
    assert _weights(lib, _cache(), length=(1 << 30) + 1) == -4


def _evict(lib, cache, lens=FAKE, now=FAKE, B=3, keep=4, recent=1, w=FAKE, wo=FAKE, p=FAKE, po=FAKE, length=8,
           new=FAKE, ws=FAKE, ws_bytes=None, st=FAKE):
    f = lib.dspark_kv_evict
    f.restype = ctypes.c_int
    need = lib.dspark_kv_evict_workspace_bytes
    need.restype = ctypes.c_size_t
    n = need(3, 2, 8) if ws_bytes is None else ws_bytes
    return f(None if cache is None else ctypes.byref(cache), lens, now, B, keep, recent, w, wo, p, po, length, new,
             ws, ctypes.c_size_t(n), st, None)


def test_evict_checks(lib):  # noqa: F811
    assert _evict(lib, None) == -1
    for bad in BAD_CACHES:
        assert _evict(lib, _cache(**bad)) == -1, bad
    for bad in (dict(lens=None), dict(now=None), dict(w=None), dict(wo=None), dict(p=None), dict(po=None),
                dict(new=None), dict(st=None), dict(B=0), dict(B=4), dict(keep=0), dict(recent=-1), dict(recent=5),
                dict(length=0), dict(wo=ctypes.c_void_p(FAKE.value + 8)), dict(po=ctypes.c_void_p(FAKE.value + 8))):
        assert _evict(lib, _cache(), **bad) == -1, bad
    assert _evict(lib, _cache(head_dim=7)) == -4
    assert _evict(lib, _cache(), length=(1 << 30) + 1, ws_bytes=1 << 50) == -4
    assert _evict(lib, _cache(), ws=None) == -2
    assert _evict(lib, _cache(), ws=ctypes.c_void_p(0x10010)) == -2
    assert _evict(lib, _cache(), ws_bytes=8) == -2


@pytest.mark.parametrize("B,H,n,ok", [(1, 1, 1, True), (32, 8, 8192, True), (0, 1, 1, False), (1, 0, 1, False),
                                      (1, 1, 0, False)])
def test_evict_workspace(lib, B, H, n, ok):  # noqa: F811
    f = lib.dspark_kv_evict_workspace_bytes
    f.restype = ctypes.c_size_t
    assert (f(B, H, n) > 0) == ok and f(B, H, n) % 256 == 0


def _at(elements):
    return ctypes.c_void_p(0x100000 + 2 * elements)


@pytest.mark.parametrize("out", [
    dict(qo=_at(1), lqo=768, hso=192),  # the parts themselves, an element on
    dict(qo=_at(192), lqo=768, hso=192),  # the next head's
    dict(qo=_at(-192 + 63), lqo=768, hso=192),
    dict(qo=_at(4 * 768 + 63), lqo=768, hso=192),  # the last row's
    dict(qo=_at(0), lqo=2304, hso=576),  # the same begin, other strides
    dict(qo=_at(0), lqo=768, hso=64),
    dict(qo=_at(64), lqo=1536, hso=192),  # between the parts, in rows of another stride
])
def test_append_query_outputs_over_a_part_of_the_queries(lib, out):  # noqa: F811
    assert _append(lib, _latent(), q=_at(0), rows=5, **out) == -1


def test_append_query_outputs_of_one_row(lib):  # noqa: F811
    """(the row stride says nothing then)"""
    assert _append(lib, _latent(), q=_at(0), rows=1, qo=_at(3 * 192 + 63), lqo=2304, hso=192) == -1
    assert _append(lib, _latent(), q=_at(0), rows=1, hq=1, qo=_at(1), lqo=2304, hso=576) == -1


@pytest.mark.parametrize("name,ld", [("q", 768), ("k", 1024), ("v", 1024), ("s", 64)])
def test_prompt_output_over_an_input(lib, name, ld):  # noqa: F811
    """7 rows of queries, 9 of keys and values: the output shares its last element with the
    first of an input, or its first with the last."""
    rows, span = (7, 768) if name == "q" else (9, 64 if name == "s" else 3 * 256 + 128)
    far = {x: ctypes.c_void_p(1 << 40 | i << 30) for i, x in enumerate(("q", "k", "v", "s"), 1)}
    # (and in the middle: of keys and values between two heads, over the second)
    for at in (-(7 * 512 - 1), (rows - 1) * ld + span - 1, 130 if name in "kv" else 3):
        assert _prompt(lib, rows=7, **{**far, name: _at(0)}, out=_at(at)) == -1, at
