"""Thin Python binding of libdspark.so (include/dspark.h).

Argument marshalling only: every function here forwards device pointers,
sizes and the current CUDA stream to the C entry point of the same name, and
raises :class:`DsparkError` on a non-zero return code.  PyTorch provides the
device buffers and the stream; every step of the computation runs in the
library's CUDA kernels.  There is no fallback: if the library is missing the
import of a function raises.
"""

from __future__ import annotations

import ctypes
import os
import threading

import torch

from . import build as _build

DSPARK_OK = 0
DSPARK_ERR_INVALID_ARG = -1
DSPARK_ERR_WORKSPACE = -2
DSPARK_ERR_CUDA = -3
DSPARK_ERR_UNSUPPORTED = -4

STATUS_CAPACITY = 1
STATUS_TOKEN_RANGE = 2
STATUS_NAN_LOGIT = 4
STATUS_BAD_INPUT = 8
STATUS_BAD_LEN = 16
STATUS_BAD_COST = 32
STATUS_INFEASIBLE = 64
STATUS_BAD_INDEX = 128
STATUS_TIMEOUT = 256
STATUS_BAD_TIER = 512
STATUS_OUT_OF_BOUNDS = 1024  # only the bounds-checked library sets it

# cost tables of at most SELECT_MAX_ENTRIES entries take the planner's
# single-CTA select path, larger ones up to DENSE_MAX_ENTRIES its single-CTA
# dense path, interpolated tables of at most INTERP_MAX_SAMPLES samples its
# single-CTA interp path (all three with the pack fused in); the rest the
# multi-CTA rank path
SELECT_MAX_ENTRIES = 31
DENSE_MAX_ENTRIES = 6143
INTERP_MAX_SAMPLES = 2048
COST_SPS_1D = 0
COST_ADDITIVE = 1
COST_ADDITIVE_INTERP = 2
DTYPE_BF16 = 0
DTYPE_F32 = 1
DTYPE_E4M3 = 2
MAX_WINDOW = 32
MAX_TIERS = 64


def planner_path(n_candidates: int, cost_kind: int, n_entries: int) -> str:
    """Which planner kernel a call takes: "select", "dense", "interp" or "rank"."""
    if cost_kind == COST_ADDITIVE_INTERP:
        return "interp" if n_entries <= INTERP_MAX_SAMPLES else "rank"
    if n_entries <= SELECT_MAX_ENTRIES:
        return "select"
    return "dense" if n_entries <= DENSE_MAX_ENTRIES else "rank"


class DsparkError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {dspark_strerror(code)} ({code})")
        self.code = code


class dspark_plan_params(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("gamma", ctypes.c_int32),
                ("survival_eps", ctypes.c_float), ("min_verify_len", ctypes.c_int32),
                ("max_verify_len", ctypes.c_int32), ("forced_budget", ctypes.c_int32)]


class dspark_cost_table(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("n", ctypes.c_int32), ("M", ctypes.c_void_p),
                ("val", ctypes.c_void_p), ("bias_ms", ctypes.c_double),
                ("alpha_ms", ctypes.c_double)]


class dspark_plan_options(ctypes.Structure):
    _fields_ = [("conf_generation", ctypes.c_void_p), ("req_generation", ctypes.c_void_p),
                ("lagged_conf_logits", ctypes.c_void_p), ("align_to_tiers", ctypes.c_int32),
                ("host_tiers", ctypes.POINTER(ctypes.c_int32)), ("n_tiers", ctypes.c_int32)]


class dspark_kv_cache(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("n_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("n_requests", ctypes.c_int32),
                ("table_width", ctypes.c_int32), ("page_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("block_table", ctypes.c_void_p)]


class dspark_norm_rope(ctypes.Structure):
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("cos_sin", ctypes.c_void_p), ("n_pos", ctypes.c_int32),
                ("rope_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


_lock = threading.Lock()
_lib = None

_VP, _I32, _I64, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t

_SIGS = {
    "dspark_strerror": (ctypes.c_char_p, [ctypes.c_int]),
    "dspark_version": (ctypes.c_int, []),
    "dspark_checked_build": (ctypes.c_int, []),
    "dspark_plan_workspace_bytes": (_SZ, [_I32, _I32]),
    "dspark_plan": (ctypes.c_int, [_VP, _VP, ctypes.POINTER(dspark_plan_params),
                                   ctypes.POINTER(dspark_cost_table), _VP, _VP, _VP, _VP, _VP,
                                   _SZ, _VP, _VP]),
    "dspark_pack_verify": (ctypes.c_int, [_VP, _VP, _VP, _VP, _I32, _I32,
                                          ctypes.POINTER(ctypes.c_int32), _I32, _I32, _VP, _VP,
                                          _VP, _VP, _VP, _VP, _VP, _VP]),
    "dspark_plan_ex": (ctypes.c_int, [_VP, _VP, ctypes.POINTER(dspark_plan_params),
                                      ctypes.POINTER(dspark_cost_table),
                                      ctypes.POINTER(dspark_plan_options), _VP, _VP, _VP, _VP, _VP,
                                      _SZ, _VP, _VP]),
    "dspark_plan_pack_ex": (ctypes.c_int, [_VP, _VP, ctypes.POINTER(dspark_plan_params),
                                           ctypes.POINTER(dspark_cost_table),
                                           ctypes.POINTER(dspark_plan_options), _VP, _VP, _VP, _VP,
                                           _VP, _VP, _VP, ctypes.POINTER(ctypes.c_int32), _I32,
                                           _I32, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP, _VP]),
    "dspark_plan_pack": (ctypes.c_int, [_VP, _VP, ctypes.POINTER(dspark_plan_params),
                                        ctypes.POINTER(dspark_cost_table), _VP, _VP, _VP, _VP,
                                        _VP, _VP, _VP, ctypes.POINTER(ctypes.c_int32), _I32, _I32,
                                        _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP, _VP]),
    "dspark_scatter_compact_to_strided": (ctypes.c_int, [_VP, _I64, _I32, _I32, _VP, _VP, _I32,
                                                         _VP, _I64, _I32, _VP, _VP]),
    "dspark_pad_to_tier": (ctypes.c_int, [_VP, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _VP]),
    "dspark_scatter_compact_to_strided_ex": (ctypes.c_int, [_VP, _I64, _I32, _I32, _VP, _VP,
                                                            _I32, _VP, _I64, _I32, _I64, _VP,
                                                            _VP]),
    "dspark_sampling_workspace_bytes": (_SZ, [_I32, _I32, _I32]),
    "dspark_sampling_accept": (ctypes.c_int, [_VP, _I32, _I64, _I32, _I32, _VP, _VP, _I64, _VP,
                                              _VP, _I32, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                                              _VP, _SZ, _VP, _VP]),
    "dspark_sampling_accept_ex": (ctypes.c_int, [_VP, _I32, _I64, _I32, _I32, _VP, _VP, _I64,
                                                 _VP, _VP, _VP, _I32, _I32, _VP, _VP, _VP, _VP,
                                                 _VP, _VP, _VP, _VP, _SZ, _VP, _VP]),
    "dspark_accept_workspace_bytes": (_SZ, [_I32, _I32]),
    "dspark_greedy_accept": (ctypes.c_int, [_VP, _I32, _I64, _I32, _I32, _VP, _VP, _VP, _I32,
                                            _I32, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP,
                                            _VP]),
    "dspark_cap_accept": (ctypes.c_int, [_VP, _I32, _I64, _I32, _VP, _VP, _VP, _I32, _I32, _VP,
                                         _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP, _VP]),
    "dspark_greedy_accept_static": (ctypes.c_int, [_VP, _I32, _I64, _I32, _I32, _VP, _VP, _VP,
                                                   _I32, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                                                   _VP]),
    "dspark_sts_confidence": (ctypes.c_int, [_VP, _VP, _I64, _I32, _VP, _VP, _VP]),
    "dspark_sts_record": (ctypes.c_int, [_VP, _VP, _VP, _VP, _I32, _I32, _VP, _VP, _VP, _I64,
                                         _VP, _VP, _VP, _VP]),
    "dspark_calibration_workspace_bytes": (_SZ, [_I32, _I32]),
    "dspark_calibration_stats": (ctypes.c_int, [_VP, _VP, _VP, _I64, _I32, _VP, _I32, _VP, _VP,
                                                _VP, _SZ, _VP, _VP]),
    "dspark_sts_fit_workspace_bytes": (_SZ, [_I64, _I32, _I32]),
    "dspark_sts_fit": (ctypes.c_int, [_VP, _VP, _VP, _I64, _I32, ctypes.POINTER(ctypes.c_float),
                                      _I32, _I32, _VP, _VP, _VP, _VP, _VP, _SZ, _VP, _VP]),
    "dspark_qk_norm_rope": (ctypes.c_int, [_VP, _I64, _VP, _I64, _I32, _I32, _I32, _I32,
                                           ctypes.POINTER(dspark_norm_rope), _VP, _VP, _I32, _VP,
                                           _I64, _VP, _I64, _VP, _VP]),
    "dspark_kv_append": (ctypes.c_int, [_VP, _I64, _VP, _I64, _VP, _I64, _I32, _I32,
                                        ctypes.POINTER(dspark_kv_cache),
                                        ctypes.POINTER(dspark_norm_rope), _VP, _VP, _VP, _VP,
                                        _I32, _VP, _I64, _VP, _VP]),
    "dspark_kv_read": (ctypes.c_int, [ctypes.POINTER(dspark_kv_cache), _VP, _VP, _I32, _I32, _I32,
                                      _VP, _VP, _I64, _VP, _VP]),
    "dspark_tree_attention_workspace_bytes": (_SZ, [_I32, _I32]),
    "dspark_tree_attention": (ctypes.c_int, [_VP, _I64, _I32, _I32, _I32, _VP, _VP, _I32, _VP,
                                             ctypes.c_float, ctypes.POINTER(dspark_kv_cache),
                                             _VP, _I64, _VP, _VP, _SZ, _VP, _VP]),
}


def library_path() -> str:
    """The normal library, or the bounds-checked one when DSPARK_CHECKED=1."""
    if os.environ.get("DSPARK_CHECKED", "0") == "1":
        return _build.CHECKED_LIB_PATH
    return _build.LIB_PATH


def load() -> ctypes.CDLL:
    """Load libdspark.so; raise if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise RuntimeError(
                    f"{os.path.basename(path)} not found at {path}: build it first "
                    "(python -c 'import __graft_entry__ as g; g.build()')")
            lib = ctypes.CDLL(path)
            for name, (res, args) in _SIGS.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


def _p(t: torch.Tensor | None, dtype: torch.dtype | None = None, name: str = "") -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:  # the current stream's handle, without the object around it
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(fn: str, rc: int) -> None:
    if rc != DSPARK_OK:
        raise DsparkError(fn, rc)


# ------------------------------------------------------------------- calls

def dspark_strerror(code: int) -> str:
    return load().dspark_strerror(int(code)).decode()


def dspark_version() -> int:
    return int(load().dspark_version())


def dspark_checked_build() -> bool:
    return bool(load().dspark_checked_build())


def dspark_plan_workspace_bytes(B: int, gamma: int) -> int:
    return int(load().dspark_plan_workspace_bytes(B, gamma))


def dspark_accept_workspace_bytes(max_rows: int, V: int) -> int:
    return int(load().dspark_accept_workspace_bytes(max_rows, V))


def dspark_plan(conf_logits, sts_temps, *, B, gamma, survival_eps, min_verify_len,
                max_verify_len, forced_budget, cost_kind, cost_M, cost_val, bias_ms=0.0,
                alpha_ms=0.0, survivals, verify_lens, budget, tau_theta, status,
                workspace, stream=None) -> None:
    """Planner: STS survivals -> budget -> verify_lens (all outputs on device).
    ``workspace``: a device byte buffer of dspark_plan_workspace_bytes(B, gamma)."""
    params = dspark_plan_params(B, gamma, survival_eps, min_verify_len, max_verify_len,
                                forced_budget)
    cost = dspark_cost_table(cost_kind, int(cost_M.numel()), _p(cost_M, torch.int32, "cost_M"),
                             _p(cost_val, torch.float64, "cost_val"), bias_ms, alpha_ms)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().dspark_plan(
        _p(conf_logits, torch.float32, "conf_logits"), _p(sts_temps, torch.float32, "sts_temps"),
        ctypes.byref(params), ctypes.byref(cost), _p(survivals, torch.float32, "survivals"),
        _p(verify_lens, torch.int32, "verify_lens"), _p(budget, torch.int32, "budget"),
        _p(tau_theta, torch.float64, "tau_theta"), _p(workspace), ws_bytes,
        _p(status, torch.int32, "status"), _stream(stream))
    _check("dspark_plan", rc)


def dspark_pack_verify(anchor, draft, prefix_lens, verify_lens, *, B, gamma, tiers, capacity,
                       packed_ids, packed_pos, packed_req, packed_src, cu_seqlens, totals,
                       status, stream=None) -> None:
    """Front-pack the verify rows; ``tiers`` is a host sequence of ints."""
    tiers = [int(t) for t in tiers]
    arr = (ctypes.c_int32 * max(1, len(tiers)))(*tiers)
    rc = load().dspark_pack_verify(
        _p(anchor, torch.int32, "anchor"), _p(draft, torch.int32, "draft"),
        _p(prefix_lens, torch.int32, "prefix_lens"), _p(verify_lens, torch.int32, "verify_lens"),
        B, gamma, arr, len(tiers), capacity, _p(packed_ids, torch.int32, "packed_ids"),
        _p(packed_pos, torch.int32, "packed_pos"), _p(packed_req, torch.int32, "packed_req"),
        _p(packed_src, torch.int32, "packed_src"), _p(cu_seqlens, torch.int32, "cu_seqlens"),
        _p(totals, torch.int32, "totals"), _p(status, torch.int32, "status"), _stream(stream))
    _check("dspark_pack_verify", rc)


def plan_options(conf_generation=None, req_generation=None, lagged_conf_logits=None,
                 align_tiers=None):
    """A dspark_plan_options (kept alive by the returned tuple's second item)
    from device tensors and a host tier list; None when no option is set."""
    if conf_generation is None and req_generation is None and lagged_conf_logits is None \
            and not align_tiers:
        return None, None
    tiers = [int(t) for t in (align_tiers or [])]
    arr = (ctypes.c_int32 * max(1, len(tiers)))(*tiers)
    opt = dspark_plan_options(_p(conf_generation, torch.int32, "conf_generation"),
                              _p(req_generation, torch.int32, "req_generation"),
                              _p(lagged_conf_logits, torch.float32, "lagged_conf_logits"),
                              1 if tiers else 0, arr, len(tiers))
    return opt, arr


def dspark_plan_ex(conf_logits, sts_temps, *, B, gamma, survival_eps, min_verify_len,
                   max_verify_len, forced_budget, cost_kind, cost_M, cost_val, bias_ms=0.0,
                   alpha_ms=0.0, survivals, verify_lens, budget, tau_theta, status, workspace,
                   conf_generation=None, req_generation=None, lagged_conf_logits=None,
                   align_tiers=None, stream=None) -> None:
    """dspark_plan with the planner options (generation mask, lagged-
    confidence budget, graph-tier alignment to ``align_tiers``)."""
    params = dspark_plan_params(B, gamma, survival_eps, min_verify_len, max_verify_len,
                                forced_budget)
    cost = dspark_cost_table(cost_kind, int(cost_M.numel()), _p(cost_M, torch.int32, "cost_M"),
                             _p(cost_val, torch.float64, "cost_val"), bias_ms, alpha_ms)
    opt, _keep = plan_options(conf_generation, req_generation, lagged_conf_logits, align_tiers)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().dspark_plan_ex(
        _p(conf_logits, torch.float32, "conf_logits"), _p(sts_temps, torch.float32, "sts_temps"),
        ctypes.byref(params), ctypes.byref(cost), None if opt is None else ctypes.byref(opt),
        _p(survivals, torch.float32, "survivals"), _p(verify_lens, torch.int32, "verify_lens"),
        _p(budget, torch.int32, "budget"), _p(tau_theta, torch.float64, "tau_theta"),
        _p(workspace), ws_bytes, _p(status, torch.int32, "status"), _stream(stream))
    _check("dspark_plan_ex", rc)


def dspark_plan_pack(conf_logits, sts_temps, anchor, draft, prefix_lens, *, B, gamma,
                     survival_eps, min_verify_len, max_verify_len, forced_budget, cost_kind,
                     cost_M, cost_val, bias_ms=0.0, alpha_ms=0.0, tiers, capacity, survivals,
                     verify_lens, budget, tau_theta, packed_ids, packed_pos, packed_req,
                     packed_src, cu_seqlens, totals, status, workspace, conf_generation=None,
                     req_generation=None, lagged_conf_logits=None, align_to_tiers=False,
                     stream=None) -> None:
    """dspark_plan then dspark_pack_verify on its verify_lens, in fewer launches
    (the pack runs inside the planner's last kernel for tables of <= 31
    entries).  The planner options as in dspark_plan_ex; alignment uses the
    pack's ``tiers``."""
    params = dspark_plan_params(B, gamma, survival_eps, min_verify_len, max_verify_len,
                                forced_budget)
    cost = dspark_cost_table(cost_kind, int(cost_M.numel()), _p(cost_M, torch.int32, "cost_M"),
                             _p(cost_val, torch.float64, "cost_val"), bias_ms, alpha_ms)
    tiers = [int(t) for t in tiers]
    arr = (ctypes.c_int32 * max(1, len(tiers)))(*tiers)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    opt, _keep = plan_options(conf_generation, req_generation, lagged_conf_logits,
                              tiers if align_to_tiers else None)
    rc = load().dspark_plan_pack_ex(
        _p(conf_logits, torch.float32, "conf_logits"), _p(sts_temps, torch.float32, "sts_temps"),
        ctypes.byref(params), ctypes.byref(cost), None if opt is None else ctypes.byref(opt),
        _p(survivals, torch.float32, "survivals"),
        _p(verify_lens, torch.int32, "verify_lens"), _p(budget, torch.int32, "budget"),
        _p(tau_theta, torch.float64, "tau_theta"), _p(anchor, torch.int32, "anchor"),
        _p(draft, torch.int32, "draft"), _p(prefix_lens, torch.int32, "prefix_lens"), arr,
        len(tiers), capacity, _p(packed_ids, torch.int32, "packed_ids"),
        _p(packed_pos, torch.int32, "packed_pos"), _p(packed_req, torch.int32, "packed_req"),
        _p(packed_src, torch.int32, "packed_src"), _p(cu_seqlens, torch.int32, "cu_seqlens"),
        _p(totals, torch.int32, "totals"), _p(workspace), ws_bytes,
        _p(status, torch.int32, "status"), _stream(stream))
    _check("dspark_plan_pack", rc)


def dspark_scatter_compact_to_strided(src, packed_src, totals, dst, *, status,
                                      wait_limit_ns=None, stream=None) -> None:
    """Copy packed row i < totals[0] of ``src`` [max_rows, width] to row
    packed_src[i] of ``dst`` [B*(gamma+1), >= width] (2-D, same dtype:
    bfloat16, float16 or float32, unit inner stride).  ``wait_limit_ns``
    (dspark_scatter_compact_to_strided_ex) bounds one pipeline wait of the
    TMA path; None keeps the 200 ms default."""
    for name, t in (("src", src), ("dst", dst)):
        if not t.is_cuda or t.dim() != 2 or t.stride(1) != 1:
            raise ValueError(f"{name}: expected a 2-D CUDA tensor with unit inner stride")
    if src.dtype != dst.dtype or src.element_size() not in (2, 4):
        raise ValueError("src and dst: same dtype of 2 or 4 bytes")
    args = (src.data_ptr(), src.stride(0), src.size(1), src.element_size(),
            _p(packed_src, torch.int32, "packed_src"), _p(totals, torch.int32, "totals"),
            src.size(0), dst.data_ptr(), dst.stride(0), dst.size(0))
    if wait_limit_ns is None:
        name = "dspark_scatter_compact_to_strided"
        rc = load().dspark_scatter_compact_to_strided(*args, _p(status, torch.int32, "status"),
                                                      _stream(stream))
    else:
        name = "dspark_scatter_compact_to_strided_ex"
        rc = load().dspark_scatter_compact_to_strided_ex(*args, int(wait_limit_ns),
                                                         _p(status, torch.int32, "status"),
                                                         _stream(stream))
    _check(name, rc)


def dspark_pad_to_tier(pad_to, *, packed_ids, packed_pos, packed_req, packed_src, totals,
                       status, capacity=None, stream=None) -> None:
    """Pad one rank's packed window to the verify tier the data-parallel
    ranks share (``pad_to``: device int32 [1], may be ``totals[1:2]``)."""
    capacity = packed_ids.numel() if capacity is None else capacity
    rc = load().dspark_pad_to_tier(
        _p(pad_to, torch.int32, "pad_to"), int(capacity), _p(packed_ids, torch.int32, "packed_ids"),
        _p(packed_pos, torch.int32, "packed_pos"), _p(packed_req, torch.int32, "packed_req"),
        _p(packed_src, torch.int32, "packed_src"), _p(totals, torch.int32, "totals"),
        _p(status, torch.int32, "status"), _stream(stream))
    _check("dspark_pad_to_tier", rc)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return DTYPE_BF16
    if t.dtype == torch.float32:
        return DTYPE_F32
    raise ValueError(f"logits: expected bfloat16 or float32, got {t.dtype}")


def _logits_ptr(logits: torch.Tensor, V: int) -> tuple[int, int]:
    """Device or pinned host logits: pinned host memory is device-accessible
    at the same address (unified addressing), and the kernels then read it
    over the host link."""
    if not (logits.is_cuda or logits.is_pinned()) or logits.dim() != 2 or logits.stride(1) != 1:
        raise ValueError("logits: expected a 2-D CUDA or pinned tensor with unit column stride")
    if logits.size(1) < V:
        raise ValueError("logits: fewer columns than V")
    return logits.data_ptr(), logits.stride(0)


def dspark_greedy_accept(logits, *, V, cu_seqlens, draft, prefix_lens, B, gamma, num_accepted,
                         bonus, commit_lens, out_tokens, workspace, status, argmax=None,
                         new_seq_lens=None, max_rows=None, stream=None) -> None:
    """Compact-mode greedy accept over the packed rows of ``logits``."""
    ptr, ld = _logits_ptr(logits, V)
    max_rows = logits.size(0) if max_rows is None else max_rows
    rc = load().dspark_greedy_accept(
        ptr, _dtype_code(logits), ld, V, max_rows, _p(cu_seqlens, torch.int32, "cu_seqlens"),
        _p(draft, torch.int32, "draft"), _p(prefix_lens, torch.int32, "prefix_lens"), B, gamma,
        _p(argmax, torch.int32, "argmax"), _p(num_accepted, torch.int32, "num_accepted"),
        _p(bonus, torch.int32, "bonus"), _p(commit_lens, torch.int32, "commit_lens"),
        _p(new_seq_lens, torch.int32, "new_seq_lens"), _p(out_tokens, torch.int32, "out_tokens"),
        _p(workspace), workspace.numel() * workspace.element_size(),
        _p(status, torch.int32, "status"), _stream(stream))
    _check("dspark_greedy_accept", rc)


def dspark_sampling_workspace_bytes(max_rows: int, B: int, gamma: int) -> int:
    return int(load().dspark_sampling_workspace_bytes(max_rows, B, gamma))


def dspark_sampling_accept(logits, draft_logits, *, V, cu_seqlens, draft, prefix_lens, B, gamma,
                           u_accept, u_bonus, num_accepted, bonus, commit_lens, out_tokens,
                           workspace, status, new_seq_lens=None, max_rows=None,
                           draft_lse=None, stream=None) -> None:
    """Speculative sampling accept: packed target rows ``logits`` and the
    draft's proposal rows ``draft_logits`` [B*gamma, >= V] (same dtype);
    ``u_accept`` [B, gamma] and ``u_bonus`` [B] are fp32 uniforms.  With
    ``draft_lse`` ([B*gamma] fp32, each draft row's log-sum-exp) the call is
    dspark_sampling_accept_ex and the draft rows are not normalised here."""
    ptr, ld = _logits_ptr(logits, V)
    dptr, dld = _logits_ptr(draft_logits, V)
    if draft_logits.dtype != logits.dtype:
        raise ValueError("draft_logits: expected the dtype of logits")
    max_rows = logits.size(0) if max_rows is None else max_rows
    if draft_lse is not None:
        rc = load().dspark_sampling_accept_ex(
            ptr, _dtype_code(logits), ld, V, max_rows, _p(cu_seqlens, torch.int32, "cu_seqlens"),
            dptr, dld, _p(draft_lse, torch.float32, "draft_lse"), _p(draft, torch.int32, "draft"),
            _p(prefix_lens, torch.int32, "prefix_lens"), B, gamma,
            _p(u_accept, torch.float32, "u_accept"), _p(u_bonus, torch.float32, "u_bonus"),
            _p(num_accepted, torch.int32, "num_accepted"), _p(bonus, torch.int32, "bonus"),
            _p(commit_lens, torch.int32, "commit_lens"),
            _p(new_seq_lens, torch.int32, "new_seq_lens"), _p(out_tokens, torch.int32, "out_tokens"),
            _p(workspace), workspace.numel() * workspace.element_size(),
            _p(status, torch.int32, "status"), _stream(stream))
        _check("dspark_sampling_accept_ex", rc)
        return
    rc = load().dspark_sampling_accept(
        ptr, _dtype_code(logits), ld, V, max_rows, _p(cu_seqlens, torch.int32, "cu_seqlens"),
        dptr, dld, _p(draft, torch.int32, "draft"), _p(prefix_lens, torch.int32, "prefix_lens"),
        B, gamma, _p(u_accept, torch.float32, "u_accept"), _p(u_bonus, torch.float32, "u_bonus"),
        _p(num_accepted, torch.int32, "num_accepted"), _p(bonus, torch.int32, "bonus"),
        _p(commit_lens, torch.int32, "commit_lens"), _p(new_seq_lens, torch.int32, "new_seq_lens"),
        _p(out_tokens, torch.int32, "out_tokens"), _p(workspace),
        workspace.numel() * workspace.element_size(), _p(status, torch.int32, "status"),
        _stream(stream))
    _check("dspark_sampling_accept", rc)


def dspark_cap_accept(logits, *, V, verify_lens, draft, prefix_lens, B, gamma, num_accepted,
                      bonus, commit_lens, out_tokens, ceiling, totals, workspace, status,
                      argmax=None, new_seq_lens=None, stream=None) -> None:
    """cap-accept over the strided [B*(gamma+1), V] verify rows."""
    ptr, ld = _logits_ptr(logits, V)
    rc = load().dspark_cap_accept(
        ptr, _dtype_code(logits), ld, V, _p(verify_lens, torch.int32, "verify_lens"),
        _p(draft, torch.int32, "draft"), _p(prefix_lens, torch.int32, "prefix_lens"), B, gamma,
        _p(argmax, torch.int32, "argmax"), _p(num_accepted, torch.int32, "num_accepted"),
        _p(bonus, torch.int32, "bonus"), _p(commit_lens, torch.int32, "commit_lens"),
        _p(new_seq_lens, torch.int32, "new_seq_lens"), _p(out_tokens, torch.int32, "out_tokens"),
        _p(ceiling, torch.int32, "ceiling"), _p(totals, torch.int32, "totals"), _p(workspace),
        workspace.numel() * workspace.element_size(), _p(status, torch.int32, "status"),
        _stream(stream))
    _check("dspark_cap_accept", rc)


def workspace(nbytes: int, device=None) -> torch.Tensor:
    """A zero-filled device byte buffer usable as a workspace (256-byte
    aligned by the caching allocator).  The planner's workspace must start
    out zero; the accept workspaces need not, but zeroing is done once, at
    allocation, off the step."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device or "cuda")


STATIC_MAX_ROWS = 32768


def dspark_greedy_accept_static(logits, *, V, cu_seqlens, draft, prefix_lens, B, gamma,
                                num_accepted, bonus, commit_lens, out_tokens, status,
                                argmax=None, new_seq_lens=None, max_rows=None,
                                stream=None) -> None:
    """dspark_greedy_accept for callers that cannot allocate device memory:
    the scratch is a library-owned device array (at most STATIC_MAX_ROWS
    rows).  Calls that overlap on the GPU race on that array."""
    ptr, ld = _logits_ptr(logits, V)
    max_rows = logits.size(0) if max_rows is None else max_rows
    rc = load().dspark_greedy_accept_static(
        ptr, _dtype_code(logits), ld, V, max_rows, _p(cu_seqlens, torch.int32, "cu_seqlens"),
        _p(draft, torch.int32, "draft"), _p(prefix_lens, torch.int32, "prefix_lens"), B, gamma,
        _p(argmax, torch.int32, "argmax"), _p(num_accepted, torch.int32, "num_accepted"),
        _p(bonus, torch.int32, "bonus"), _p(commit_lens, torch.int32, "commit_lens"),
        _p(new_seq_lens, torch.int32, "new_seq_lens"), _p(out_tokens, torch.int32, "out_tokens"),
        _p(status, torch.int32, "status"), _stream(stream))
    _check("dspark_greedy_accept_static", rc)


# -------------------------------------------------------------- calibration

def dspark_sts_confidence(conf_logits, *, sts_temps, conf_out, status, stream=None) -> None:
    """c = sigmoid(z / T) elementwise over conf_logits [n_rows, gamma]."""
    n_rows, gamma = conf_logits.shape
    rc = load().dspark_sts_confidence(
        _p(conf_logits, torch.float32, "conf_logits"), _p(sts_temps, torch.float32, "sts_temps"),
        n_rows, gamma, _p(conf_out, torch.float32, "conf_out"), _p(status, torch.int32, "status"),
        _stream(stream))
    _check("dspark_sts_confidence", rc)


def dspark_sts_record(conf_logits, *, num_correct, B, gamma, rec_logits, rec_correct, rec_tested,
                      cursor, status, verify_lens=None, select=None, prefix_mask=None,
                      stream=None) -> None:
    """Append the selected requests of one step to the recorded-sample ring
    (rec_logits [capacity, gamma] fp32, rec_correct / rec_tested [capacity]
    int32) at the device cursor (an int64 [1] tensor, bit-identical to the
    C ABI's uint64)."""
    rc = load().dspark_sts_record(
        _p(conf_logits, torch.float32, "conf_logits"), _p(num_correct, torch.int32, "num_correct"),
        _p(verify_lens, torch.int32, "verify_lens"), _p(select, torch.uint8, "select"), B, gamma,
        _p(rec_logits, torch.float32, "rec_logits"), _p(rec_correct, torch.int32, "rec_correct"),
        _p(rec_tested, torch.int32, "rec_tested"), rec_correct.numel(),
        _p(cursor, torch.int64, "cursor"), _p(prefix_mask, torch.uint8, "prefix_mask"),
        _p(status, torch.int32, "status"), _stream(stream))
    _check("dspark_sts_record", rc)


def dspark_calibration_workspace_bytes(gamma: int, n_bins: int) -> int:
    return int(load().dspark_calibration_workspace_bytes(gamma, n_bins))


def dspark_calibration_stats(rec_logits, *, rec_correct, rec_tested, N, gamma, sts_temps, n_bins,
                             metrics, workspace, status, hist=None, stream=None) -> None:
    """Per-depth calibration (metrics [2, gamma, 4] fp64; hist [2, gamma,
    n_bins, 3] int64 holding the C ABI's uint64 counts)."""
    rc = load().dspark_calibration_stats(
        _p(rec_logits, torch.float32, "rec_logits"), _p(rec_correct, torch.int32, "rec_correct"),
        _p(rec_tested, torch.int32, "rec_tested"), N, gamma,
        _p(sts_temps, torch.float32, "sts_temps"), n_bins, _p(hist, torch.int64, "hist"),
        _p(metrics, torch.float64, "metrics"), _p(workspace),
        workspace.numel() * workspace.element_size(), _p(status, torch.int32, "status"),
        _stream(stream))
    _check("dspark_calibration_stats", rc)


def dspark_sts_fit_workspace_bytes(N: int, n_temps: int, n_bins: int) -> int:
    return int(load().dspark_sts_fit_workspace_bytes(N, n_temps, n_bins))


def dspark_sts_fit(rec_logits, *, rec_correct, rec_tested, N, gamma, temp_grid, n_bins,
                   sts_temps_out, choice, workspace, status, ece_curve=None, n_obs=None,
                   stream=None) -> None:
    """Sequential per-depth temperature fit over ``temp_grid`` (a host
    sequence of positive temperatures)."""
    grid = (ctypes.c_float * len(temp_grid))(*[float(t) for t in temp_grid])
    rc = load().dspark_sts_fit(
        _p(rec_logits, torch.float32, "rec_logits"), _p(rec_correct, torch.int32, "rec_correct"),
        _p(rec_tested, torch.int32, "rec_tested"), N, gamma, grid, len(temp_grid), n_bins,
        _p(sts_temps_out, torch.float32, "sts_temps_out"), _p(choice, torch.int32, "choice"),
        _p(ece_curve, torch.float64, "ece_curve"), _p(n_obs, torch.int64, "n_obs"),
        _p(workspace), workspace.numel() * workspace.element_size(),
        _p(status, torch.int32, "status"), _stream(stream))
    _check("dspark_sts_fit", rc)


# --------------------------------------------- verify window over a cache

class KVCache:
    """One layer's paged cache over tensors the caller owns (the C ABI's
    dspark_kv_cache, filled once).

    ``k``, ``v``: [n_pages, page_size, n_kv_heads, head_dim], bfloat16, float32
    or float8_e4m3fn, of the same strides with a unit inner one; tokens and
    heads may lie in either order (pass a transposed view).  ``block_table``:
    int32 [n_requests, table_width].  ``k_scale``, ``v_scale``: fp32 [n_pages,
    n_kv_heads, page_size], for float8 only.  The tensors are kept referenced."""

    def __init__(self, k, v, block_table, k_scale=None, v_scale=None):
        kinds = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32,
                 torch.float8_e4m3fn: DTYPE_E4M3}
        for name, t in (("k", k), ("v", v)):
            if not t.is_cuda or t.dim() != 4 or t.stride(3) != 1:
                raise ValueError(f"{name}: expected a 4-D CUDA tensor with unit inner stride")
        if k.dtype not in kinds or v.dtype != k.dtype:
            raise ValueError("k and v: expected one of bfloat16, float32 and float8_e4m3fn")
        if v.shape != k.shape or v.stride() != k.stride():
            raise ValueError("v: expected the shape and strides of k")
        if block_table.dim() != 2:
            raise ValueError("block_table: expected a 2-D tensor")
        n_pages, page, heads, dim = k.shape
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if (t is not None) != (k.dtype == torch.float8_e4m3fn):
                raise ValueError(f"{name}: expected with float8_e4m3fn entries, and only with them")
            if t is not None and tuple(t.shape) != (n_pages, heads, page):
                raise ValueError(f"{name}: expected shape {(n_pages, heads, page)}")
        self.k, self.v, self.block_table = k, v, block_table
        self.k_scale, self.v_scale = k_scale, v_scale
        self.n_kv_heads, self.head_dim = heads, dim
        self.desc = dspark_kv_cache(
            kinds[k.dtype], n_pages, page, heads, dim, block_table.size(0), block_table.size(1),
            k.stride(0), k.stride(1), k.stride(2), k.data_ptr(), v.data_ptr(),
            _p(k_scale, torch.float32, "k_scale"), _p(v_scale, torch.float32, "v_scale"),
            _p(block_table, torch.int32, "block_table"))
        self.ref = ctypes.byref(self.desc)


_NO_ROWS = 256  # a tensor without elements has no address; one that is never read stands for it


def _rows(t: torch.Tensor, name: str, dtype, heads: int, dim: int, rows: int) -> tuple[int, int]:
    """Pointer and row stride of [rows, heads, head_dim] rows: heads packed,
    any row stride."""
    if t.dim() != 3 or not t.is_cuda:
        raise ValueError(f"{name}: expected a 3-D CUDA tensor [rows, heads, head_dim]")
    n, h, d = t.shape
    ld, sh, sd = t.stride()
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if (sd != 1 and d > 1) or (sh != d and h > 1):
        raise ValueError(f"{name}: expected packed heads with unit inner stride")
    if h != heads or d != dim:
        raise ValueError(f"{name}: expected {heads} heads of {dim} elements, got {h} of {d}")
    if n < rows:
        raise ValueError(f"{name}: expected at least {rows} rows, got {n}")
    return t.data_ptr() if n else _NO_ROWS, ld if n > 1 else max(ld, h * d)


def _index(t, n, name):
    """Pointer of at least n contiguous int32 elements, or None."""
    if t is None:
        return None
    if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
        return _p(t, torch.int32, name)  # says what is wrong
    if t.numel() < n:
        raise ValueError(f"{name}: expected at least {n} elements, got {t.numel()}")
    return t.data_ptr() if t.numel() else _NO_ROWS


def _norm_rope(dtype, dim, q_weight, k_weight, eps, cos_sin, interleaved):
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None and w.numel() != dim:
            raise ValueError(f"{name}: expected {dim} elements")
    n_pos, rope_dim = (0, 0) if cos_sin is None else cos_sin.shape
    return dspark_norm_rope(_p(q_weight, dtype, "q_weight"), _p(k_weight, dtype, "k_weight"), eps,
                            _p(cos_sin, torch.float32, "cos_sin"), n_pos, rope_dim,
                            1 if interleaved else 0)


def dspark_qk_norm_rope(q, k, *, status, pos=None, totals=None, q_weight=None, k_weight=None,
                        eps=1e-6, cos_sin=None, interleaved=False, q_out=None, k_out=None,
                        max_rows=None, stream=None) -> None:
    """RMS norm of each head's queries and keys (where a weight is given) and
    rotation of their first cos_sin.size(1) elements (where ``cos_sin`` is:
    fp32 [n_pos, rope_dim], cosines then sines), in one pass.  ``q``, ``k``:
    [rows, heads, head_dim] bfloat16 or float32 with packed heads, either may
    be None; the outputs default to the inputs themselves (in place)."""
    first = q if q is not None else k
    if first is None:
        raise ValueError("q and k: expected at least one of them")
    dtype, dim = first.dtype, first.size(2)
    code = _dtype_code(first)
    max_rows = first.size(0) if max_rows is None else max_rows
    args = []
    for name, t, o in (("q", q, q_out), ("k", k, k_out)):
        if t is None:
            if o is not None:
                raise ValueError(f"{name}_out: expected with {name} only")
            args.append((None, 0, None, 0, 0))
            continue
        heads = t.size(1)
        args.append(_rows(t, name, dtype, heads, dim, max_rows)
                    + _rows(t if o is None else o, name + "_out", dtype, heads, dim, max_rows)
                    + (heads,))
    (qp, lq, qo, lqo, hq), (kp, lk, ko, lko, hk) = args
    nr = _norm_rope(dtype, dim, q_weight, k_weight, eps, cos_sin, interleaved)
    rc = load().dspark_qk_norm_rope(
        qp, lq, kp, lk, code, hq, hk, dim, ctypes.byref(nr), _index(pos, max_rows, "pos"),
        _index(totals, 1, "totals"), max_rows, qo, lqo, ko, lko,
        _p(status, torch.int32, "status"), _stream(stream))
    _check("dspark_qk_norm_rope", rc)


def dspark_kv_append(k, v, cache: KVCache, *, req, status, pos=None, cache_pos=None, q=None,
                     q_out=None, totals=None, q_weight=None, k_weight=None, eps=1e-6,
                     cos_sin=None, interleaved=False, max_rows=None, stream=None) -> None:
    """dspark_qk_norm_rope with the keys, and the values as they are, going
    into ``cache`` at the rows' positions (``cache_pos``, else ``pos``);
    quantised there if it holds float8.  ``q`` (with ``q_out``, in place by
    default) rides along in the same pass."""
    dtype, dim, hkv = k.dtype, cache.head_dim, cache.n_kv_heads
    code = _dtype_code(k)
    max_rows = k.size(0) if max_rows is None else max_rows
    qp = lq = qo = lqo = None
    hq = 0
    if q is None and q_out is not None:
        raise ValueError("q_out: expected with q only")
    if q is not None:
        hq = q.size(1)
        qp, lq = _rows(q, "q", dtype, hq, dim, max_rows)
        qo, lqo = _rows(q if q_out is None else q_out, "q_out", dtype, hq, dim, max_rows)
    kp, lk = _rows(k, "k", dtype, hkv, dim, max_rows)
    vp, lv = _rows(v, "v", dtype, hkv, dim, max_rows)
    nr = None
    if q_weight is not None or k_weight is not None or cos_sin is not None:
        nr = _norm_rope(dtype, dim, q_weight, k_weight, eps, cos_sin, interleaved)
    rc = load().dspark_kv_append(
        qp, lq or 0, kp, lk, vp, lv, code, hq, cache.ref, None if nr is None else ctypes.byref(nr),
        _index(req, max_rows, "req"), _index(pos, max_rows, "pos"),
        _index(cache_pos, max_rows, "cache_pos"), _index(totals, 1, "totals"), max_rows, qo,
        lqo or 0, _p(status, torch.int32, "status"), _stream(stream))
    _check("dspark_kv_append", rc)


def dspark_kv_read(cache: KVCache, *, start, cu_rows, k_out, v_out, status, max_rows=None,
                   stream=None) -> None:
    """Positions start[r], start[r]+1, ... of each request back as rows
    cu_rows[r]..cu_rows[r+1]-1 of ``k_out`` and ``v_out`` ([rows, n_kv_heads,
    head_dim], bfloat16 or float32)."""
    B = start.numel()
    max_rows = k_out.size(0) if max_rows is None else max_rows
    kp, ld = _rows(k_out, "k_out", k_out.dtype, cache.n_kv_heads, cache.head_dim, max_rows)
    vp, ldv = _rows(v_out, "v_out", k_out.dtype, cache.n_kv_heads, cache.head_dim, max_rows)
    if ldv != ld:
        raise ValueError("v_out: expected the row stride of k_out")
    rc = load().dspark_kv_read(
        cache.ref, _p(start, torch.int32, "start"), _index(cu_rows, B + 1, "cu_rows"), B,
        max_rows, _dtype_code(k_out), kp, vp, ld, _p(status, torch.int32, "status"),
        _stream(stream))
    _check("dspark_kv_read", rc)


def dspark_tree_attention_workspace_bytes(n_q_heads: int, head_dim: int) -> int:
    return int(load().dspark_tree_attention_workspace_bytes(n_q_heads, head_dim))


def dspark_tree_attention(q, cache: KVCache, *, cu_seqlens, prefix_lens, scale, out, workspace,
                          status, ancestors=None, lse=None, max_rows=None, stream=None) -> None:
    """Attention of the packed window's rows ``q`` [rows, n_q_heads, head_dim]
    over ``cache``: every position before the request's prefix length and the
    window's tokens whose bit is set in the row's ``ancestors`` word (int32
    bits [rows]; None: a chain).  ``out`` like ``q`` and beside it, not over it
    (slices of one buffer's rows will do); ``lse`` fp32 [rows, n_q_heads],
    optional."""
    hq, dim = q.size(1), cache.head_dim
    code = _dtype_code(q)
    max_rows = q.size(0) if max_rows is None else max_rows
    B = prefix_lens.numel()
    qp, lq = _rows(q, "q", q.dtype, hq, dim, max_rows)
    op, lo = _rows(out, "out", q.dtype, hq, dim, max_rows)
    if lse is not None and lse.numel() < max_rows * hq:
        raise ValueError(f"lse: expected at least {max_rows * hq} elements")
    rc = load().dspark_tree_attention(
        qp, lq, code, hq, max_rows, _index(cu_seqlens, B + 1, "cu_seqlens"),
        _p(prefix_lens, torch.int32, "prefix_lens"), B, _index(ancestors, max_rows, "ancestors"),
        scale, cache.ref, op, lo, _p(lse, torch.float32, "lse"), _p(workspace),
        workspace.numel() * workspace.element_size(), _p(status, torch.int32, "status"),
        _stream(stream))
    _check("dspark_tree_attention", rc)
