"""Python binding of libnf.so, the GB300 (sm_103a) inner-persistent row
normalization library.

Two layers, both thin:

* ``nf_*`` functions with the C ABI's names and arguments (device pointers
  as ints, a stream handle as an int).  They return the C status code.
* Tensor helpers (``fused_add_rmsnorm``, ``rmsnorm_fwd``, ``layernorm_fwd``,
  ``layernorm_bwd``) that check dtypes/devices/contiguity, take pointers and
  the current CUDA stream from PyTorch, call the C function and raise
  ``NFError`` on a non-OK status.  PyTorch only provides device memory and
  streams; every step of the computation runs in the library's kernels.

There is no fallback: if libnf.so is missing, loading raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnf.so")

NF_OK = 0
NF_ERR_INVALID_ARG = 1
NF_ERR_UNSUPPORTED_HIDDEN = 2
NF_ERR_MISALIGNED = 3
NF_ERR_WORKSPACE_TOO_SMALL = 4
NF_ERR_CUDA = 5
NF_ERR_TIMEOUT = 6
NF_ERR_UNSUPPORTED_PATH = 7

NF_PATH_AUTO, NF_PATH_REG, NF_PATH_CLUSTER, NF_PATH_BULK, NF_PATH_DYNAMIC, NF_PATH_SPLIT, \
    NF_PATH_GRID = 0, 1, 2, 3, 4, 5, 6
PATHS = {"auto": NF_PATH_AUTO, "reg": NF_PATH_REG, "cluster": NF_PATH_CLUSTER, "bulk": NF_PATH_BULK,
         "dynamic": NF_PATH_DYNAMIC, "split": NF_PATH_SPLIT, "grid": NF_PATH_GRID}
PATH_NAMES = {v: k for k, v in PATHS.items()}

NF_OP_FUSED_ADD_RMSNORM, NF_OP_RMSNORM_FWD, NF_OP_LAYERNORM_FWD, NF_OP_LAYERNORM_BWD, \
    NF_OP_RMSNORM_BWD = 0, 1, 2, 3, 4
OPS = {"fused_add_rmsnorm": 0, "rmsnorm_fwd": 1, "layernorm_fwd": 2, "layernorm_bwd": 3,
       "rmsnorm_bwd": 4}

HIDDEN_SET = (1024, 2048, 4096, 5120, 8192, 12288)   # compiled sizes
DYN_MAX_HIDDEN_FWD = 32768    # runtime-hidden path: any multiple of 8 up to these
DYN_MAX_HIDDEN_BWD = 16384
LONG_MAX_HIDDEN_FWD = 262144  # grid-parallel cluster path for longer rows
LONG_MAX_HIDDEN_BWD = 131072
SPLIT_MAX_HIDDEN = 1 << 26    # NF_SPLIT_MAX_HIDDEN: rows across any number of CTAs
Q8_MAX_HIDDEN = 32768         # NF_Q8_MAX_HIDDEN: rows with an 8-bit output
TOP_MAX = 32                  # NF_TOP_MAX: alternatives per row of token_logprob_fwd
GRID_MAX_ROWS = 8             # the grid family (rows held on chip) takes 1 to 8 rows

NF_Q8_E4M3, NF_Q8_INT8 = 0, 1
Q8_FORMATS = {"e4m3": NF_Q8_E4M3, "int8": NF_Q8_INT8}
Q8_GROUP = 128                # columns per scale of the grouped 8-bit output

NF_BF16, NF_F32 = 0, 1        # nf_dtype

HEAD_MAX_DIM = 512            # NF_HEAD_MAX_DIM: elements of an attention head
NF_ROPE_HALF, NF_ROPE_INTERLEAVED = 0, 1
ROPE_LAYOUTS = {"half": NF_ROPE_HALF, "interleaved": NF_ROPE_INTERLEAVED}
NF_ROPE_PLAIN, NF_ROPE_LINEAR, NF_ROPE_NTK, NF_ROPE_PARTS = 0, 1, 2, 3
ROPE_SCALINGS = {"plain": NF_ROPE_PLAIN, "linear": NF_ROPE_LINEAR, "ntk": NF_ROPE_NTK, "parts": NF_ROPE_PARTS}
NF_CACHE_SAME, NF_CACHE_E4M3, NF_CACHE_INT8 = 0, 1, 2

# Every symbol include/nf.h declares.
EXPORTS = (
    "nf_fused_add_rmsnorm", "nf_rmsnorm_fwd", "nf_layernorm_fwd",
    "nf_layernorm_bwd_workspace_size", "nf_layernorm_bwd",
    "nf_rmsnorm_bwd_workspace_size", "nf_rmsnorm_bwd", "nf_layernorm_bwd_noalloc",
    "nf_outer_norm_workspace_size", "nf_outer_norm_fwd", "nf_outer_norm_bwd",
    "nf_fused_add_rmsnorm_bwd", "nf_workspace_size", "nf_fused_add_rmsnorm_ws", "nf_rmsnorm_fwd_ws",
    "nf_layernorm_fwd_ws",
    "nf_rmsnorm_q8", "nf_fused_add_rmsnorm_q8",
    "nf_embedding_fwd", "nf_embedding_bwd_workspace_size", "nf_embedding_bwd",
    "nf_token_logprob_fwd", "nf_token_logprob_bwd",
    "nf_rope_rates", "nf_rope_rates_of", "nf_rope_fwd", "nf_rope_bwd",
    "nf_qk_rmsnorm_rope_fwd", "nf_qk_rmsnorm_rope_bwd_workspace_size", "nf_qk_rmsnorm_rope_bwd",
    "nf_kv_append",
    "nf_set_path", "nf_plan_query", "nf_plan_compute", "nf_get_device_status",
    "nf_selftest_wait_timeout", "nf_selftest_grid_timeout", "nf_selftest_floor", "nf_status_string",
    "nf_version",
)


class NFError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


class Plan(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int32), ("grid", ctypes.c_int32), ("block", ctypes.c_int32),
                ("cluster", ctypes.c_int32), ("rows_per_cta", ctypes.c_int32),
                ("smem_bytes", ctypes.c_int32), ("launches", ctypes.c_int32),
                ("partials", ctypes.c_int32)]

    def as_dict(self):
        d = {f: getattr(self, f) for f, _ in self._fields_}
        d["path"] = PATH_NAMES.get(d["path"], d["path"])
        return d


class Heads(ctypes.Structure):
    """nf_heads: a set of heads by its first element and its strides (in elements)."""
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("heads", ctypes.c_int32)]


class Rope(ctypes.Structure):
    """nf_rope: the rotation of a call."""
    _fields_ = [("rates", ctypes.c_void_p), ("dim", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("magnitude", ctypes.c_float), ("positions", ctypes.c_void_p),
                ("position_bytes", ctypes.c_int32), ("position_stride", ctypes.c_int64)]


class Pages(ctypes.Structure):
    """nf_pages: a paged cache of keys or values."""
    _fields_ = [("data", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("slot_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("scale", ctypes.c_void_p), ("scale_page_stride", ctypes.c_int64),
                ("scale_slot_stride", ctypes.c_int64), ("scale_head_stride", ctypes.c_int64)]


_lock = threading.Lock()
_lib = None

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_F = ctypes.c_float
_S = ctypes.c_int
_D = ctypes.c_double
_Z = ctypes.c_size_t
_I32 = ctypes.c_int32
_H = ctypes.POINTER(Heads)
_R = ctypes.POINTER(Rope)
_C = ctypes.POINTER(Pages)


def _bind(lib):
    sig = {
        "nf_fused_add_rmsnorm": (_S, [_P, _P, _P, _I64, _I64, _F, _P]),
        "nf_rmsnorm_fwd": (_S, [_P, _P, _P, _I64, _I64, _F, _P]),
        "nf_layernorm_fwd": (_S, [_P, _P, _P, _P, _P, _P, _I64, _I64, _F, _P]),
        "nf_workspace_size": (ctypes.c_size_t, [ctypes.c_int, _I64, _I64]),
        "nf_fused_add_rmsnorm_ws": (_S, [_P, _P, _P, _I64, _I64, _F, _P, ctypes.c_size_t, _P]),
        "nf_rmsnorm_fwd_ws": (_S, [_P, _P, _P, _I64, _I64, _F, _P, ctypes.c_size_t, _P]),
        "nf_layernorm_fwd_ws": (_S, [_P, _P, _P, _P, _P, _P, _I64, _I64, _F, _P, ctypes.c_size_t, _P]),
        "nf_layernorm_bwd_workspace_size": (ctypes.c_size_t, [_I64, _I64]),
        "nf_layernorm_bwd": (_S, [_P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _P, ctypes.c_size_t, _P]),
        "nf_rmsnorm_bwd_workspace_size": (ctypes.c_size_t, [_I64, _I64]),
        "nf_rmsnorm_bwd": (_S, [_P, _P, _P, _P, _P, _I64, _I64, _F, _P, ctypes.c_size_t, _P]),
        "nf_layernorm_bwd_noalloc": (_S, [_P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _P]),
        "nf_outer_norm_workspace_size": (ctypes.c_size_t, [_I64, _I64]),
        "nf_fused_add_rmsnorm_bwd": (_S, [_P, _P, _P, _P, _P, _P, _I64, _I64, _F, _P, ctypes.c_size_t, _P]),
        "nf_outer_norm_fwd": (_S, [_P, _P, _P, _P, _P, _P, _I64, _I64, _F, _P, ctypes.c_size_t, _P]),
        "nf_outer_norm_bwd": (_S, [_P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _P, ctypes.c_size_t, _P]),
        "nf_rmsnorm_q8": (_S, [_P, _P, _P, _P, _I64, _I64, _F, _S, _I64, _P]),
        "nf_fused_add_rmsnorm_q8": (_S, [_P, _P, _P, _P, _P, _I64, _I64, _F, _S, _I64, _P]),
        "nf_embedding_fwd": (_S, [_P, _P, _S, _P, _I64, _I64, _I64, _F, _P]),
        "nf_embedding_bwd_workspace_size": (ctypes.c_size_t, [_I64, _I64]),
        "nf_embedding_bwd": (_S, [_P, _S, _S, _P, _P, _S, _I64, _I64, _I64, _F, _P, ctypes.c_size_t, _P]),
        "nf_token_logprob_fwd": (_S, [_P, _P, _P, _P, _P, _P, _S, _I64, _P, _S, _I64, _I64, _F, _S, _P]),
        "nf_token_logprob_bwd": (_S, [_P, _I64, _P, _S, _I64, _P, _S, _P, _P, _P, _P, _I64, _I64, _F, _P]),
        "nf_rope_rates": (_S, [_P, _I32, _D, _S, _D, _D, _D, _D]),
        "nf_rope_rates_of": (_S, [_P, _P, _I32]),
        "nf_rope_fwd": (_S, [_H, _H, _H, _H, _S, _I64, _I64, _I64, _R, _P]),
        "nf_rope_bwd": (_S, [_H, _H, _H, _H, _S, _I64, _I64, _I64, _R, _P]),
        "nf_qk_rmsnorm_rope_fwd": (_S, [_H, _H, _P, _H, _H, _P, _S, _I64, _I64, _I64, _F, _R, _P]),
        "nf_qk_rmsnorm_rope_bwd_workspace_size": (_Z, [_I64]),
        "nf_qk_rmsnorm_rope_bwd": (_S, [_H, _P, _H, _H, _P, _H, _P, _H, _H, _P, _S, _I64, _I64, _I64, _F, _R, _P,
                                        _Z, _P]),
        "nf_kv_append": (_S, [_C, _C, _S, _I64, _I32, _H, _H, _P, _H, _H, _P, _S, _I64, _I64, _I64, _P, _P, _P, _I64,
                              _I32, _F, _R, _P]),
        "nf_set_path": (_S, [_S]),
        "nf_plan_query": (_S, [_S, _I64, _I64, ctypes.POINTER(Plan)]),
        "nf_plan_compute": (_S, [_S, _I64, _I64, ctypes.c_int32, _S, ctypes.POINTER(Plan)]),
        "nf_get_device_status": (_S, [_P]),
        "nf_selftest_wait_timeout": (_S, [_I64, _P]),
        "nf_selftest_grid_timeout": (_S, [_P, _I64, _P]),
        "nf_selftest_floor": (_S, [ctypes.c_int32, _P, _P, _I64, _P]),
        "nf_status_string": (ctypes.c_char_p, [_S]),
        "nf_version": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


def lib():
    """The loaded libnf.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with "
                    "`python -m row_normalization_inner_gb300.build` (no fallback exists)")
            _lib = _bind(ctypes.CDLL(LIB_PATH))
        return _lib


def status_string(status: int) -> str:
    return lib().nf_status_string(status).decode()


def version() -> str:
    return lib().nf_version().decode()


# ---------------------------------------------------------------- C-ABI names

def nf_fused_add_rmsnorm(x, residual, weight, rows, hidden, eps, stream) -> int:
    return lib().nf_fused_add_rmsnorm(x, residual, weight, rows, hidden, eps, stream)


def nf_rmsnorm_fwd(y, x, weight, rows, hidden, eps, stream) -> int:
    return lib().nf_rmsnorm_fwd(y, x, weight, rows, hidden, eps, stream)


def nf_workspace_size(op, rows, hidden) -> int:
    return lib().nf_workspace_size(op, rows, hidden)


def nf_fused_add_rmsnorm_ws(x, residual, weight, rows, hidden, eps, workspace, workspace_bytes,
                            stream) -> int:
    return lib().nf_fused_add_rmsnorm_ws(x, residual, weight, rows, hidden, eps, workspace,
                                         workspace_bytes, stream)


def nf_rmsnorm_fwd_ws(y, x, weight, rows, hidden, eps, workspace, workspace_bytes, stream) -> int:
    return lib().nf_rmsnorm_fwd_ws(y, x, weight, rows, hidden, eps, workspace, workspace_bytes,
                                   stream)


def nf_layernorm_fwd_ws(y, mean, rstd, x, gamma, beta, rows, hidden, eps, workspace,
                        workspace_bytes, stream) -> int:
    return lib().nf_layernorm_fwd_ws(y, mean, rstd, x, gamma, beta, rows, hidden, eps, workspace,
                                     workspace_bytes, stream)


def nf_layernorm_fwd(y, mean, rstd, x, gamma, beta, rows, hidden, eps, stream) -> int:
    return lib().nf_layernorm_fwd(y, mean, rstd, x, gamma, beta, rows, hidden, eps, stream)


def nf_layernorm_bwd_workspace_size(rows, hidden) -> int:
    return lib().nf_layernorm_bwd_workspace_size(rows, hidden)


def nf_layernorm_bwd(dx, dgamma, dbeta, dy, x, mean, rstd, gamma, rows, hidden, workspace,
                     workspace_bytes, stream) -> int:
    return lib().nf_layernorm_bwd(dx, dgamma, dbeta, dy, x, mean, rstd, gamma, rows, hidden,
                                  workspace, workspace_bytes, stream)


def nf_rmsnorm_bwd_workspace_size(rows, hidden) -> int:
    return lib().nf_rmsnorm_bwd_workspace_size(rows, hidden)


def nf_rmsnorm_bwd(dx, dw, dy, x, weight, rows, hidden, eps, workspace, workspace_bytes,
                   stream) -> int:
    return lib().nf_rmsnorm_bwd(dx, dw, dy, x, weight, rows, hidden, eps, workspace,
                                workspace_bytes, stream)


def nf_layernorm_bwd_noalloc(dx, dgamma, dbeta, dy, x, mean, rstd, gamma, rows, hidden,
                             stream) -> int:
    return lib().nf_layernorm_bwd_noalloc(dx, dgamma, dbeta, dy, x, mean, rstd, gamma, rows,
                                          hidden, stream)


NOALLOC_SCRATCH_BYTES = 16 << 20  # NF_LAYERNORM_BWD_NOALLOC_SCRATCH_BYTES


def nf_fused_add_rmsnorm_bwd(dx, dw, dy, dres, residual, weight, rows, hidden, eps, workspace,
                             workspace_bytes, stream) -> int:
    return lib().nf_fused_add_rmsnorm_bwd(dx, dw, dy, dres, residual, weight, rows, hidden, eps,
                                          workspace, workspace_bytes, stream)


def nf_outer_norm_workspace_size(rows, hidden) -> int:
    return lib().nf_outer_norm_workspace_size(rows, hidden)


def nf_outer_norm_fwd(y, mean, rstd, x, gamma, beta, rows, hidden, eps, workspace,
                      workspace_bytes, stream) -> int:
    return lib().nf_outer_norm_fwd(y, mean, rstd, x, gamma, beta, rows, hidden, eps, workspace,
                                   workspace_bytes, stream)


def nf_outer_norm_bwd(dx, dgamma, dbeta, dy, x, mean, rstd, gamma, rows, hidden, workspace,
                      workspace_bytes, stream) -> int:
    return lib().nf_outer_norm_bwd(dx, dgamma, dbeta, dy, x, mean, rstd, gamma, rows, hidden,
                                   workspace, workspace_bytes, stream)


def nf_rmsnorm_q8(q, scale, x, weight, rows, hidden, eps, format, group, stream) -> int:
    return lib().nf_rmsnorm_q8(q, scale, x, weight, rows, hidden, eps, format, group, stream)


def nf_fused_add_rmsnorm_q8(q, scale, x, residual, weight, rows, hidden, eps, format, group,
                            stream) -> int:
    return lib().nf_fused_add_rmsnorm_q8(q, scale, x, residual, weight, rows, hidden, eps, format,
                                         group, stream)


def nf_embedding_fwd(y, ids, id_bytes, table, tokens, vocab, hidden, scale, stream) -> int:
    return lib().nf_embedding_fwd(y, ids, id_bytes, table, tokens, vocab, hidden, scale, stream)


def nf_embedding_bwd_workspace_size(tokens, hidden) -> int:
    return lib().nf_embedding_bwd_workspace_size(tokens, hidden)


def nf_embedding_bwd(dtable, dtable_type, accumulate, dy, ids, id_bytes, tokens, vocab, hidden, scale,
                     workspace, workspace_bytes, stream) -> int:
    return lib().nf_embedding_bwd(dtable, dtable_type, accumulate, dy, ids, id_bytes, tokens, vocab,
                                  hidden, scale, workspace, workspace_bytes, stream)


def nf_token_logprob_fwd(logprob, entropy, stats, top_logprob, top_ids, logits, type, stride, targets,
                         id_bytes, rows, vocab, temperature, top, stream) -> int:
    return lib().nf_token_logprob_fwd(logprob, entropy, stats, top_logprob, top_ids, logits, type,
                                      stride, targets, id_bytes, rows, vocab, temperature, top, stream)


def nf_token_logprob_bwd(dlogits, dstride, logits, type, stride, targets, id_bytes, stats, entropy,
                         d_logprob, d_entropy, rows, vocab, temperature, stream) -> int:
    return lib().nf_token_logprob_bwd(dlogits, dstride, logits, type, stride, targets, id_bytes, stats,
                                      entropy, d_logprob, d_entropy, rows, vocab, temperature, stream)


def nf_rope_rates(rates, dim, base, scaling, factor, length, low, high) -> int:
    return lib().nf_rope_rates(rates, dim, base, scaling, factor, length, low, high)


def nf_rope_rates_of(rates, frequencies, count) -> int:
    return lib().nf_rope_rates_of(rates, frequencies, count)


# The entry points on heads take Heads, Rope and Pages structures (None for a null pointer).

def nf_rope_fwd(q_out, q, k_out, k, type, batch, tokens, head_dim, rope, stream) -> int:
    return lib().nf_rope_fwd(q_out, q, k_out, k, type, batch, tokens, head_dim, rope, stream)


def nf_rope_bwd(dq, dq_out, dk, dk_out, type, batch, tokens, head_dim, rope, stream) -> int:
    return lib().nf_rope_bwd(dq, dq_out, dk, dk_out, type, batch, tokens, head_dim, rope, stream)


def nf_qk_rmsnorm_rope_fwd(q_out, q, q_weight, k_out, k, k_weight, type, batch, tokens, head_dim, eps, rope,
                           stream) -> int:
    return lib().nf_qk_rmsnorm_rope_fwd(q_out, q, q_weight, k_out, k, k_weight, type, batch, tokens, head_dim, eps,
                                        rope, stream)


def nf_qk_rmsnorm_rope_bwd_workspace_size(head_dim) -> int:
    return lib().nf_qk_rmsnorm_rope_bwd_workspace_size(head_dim)


def nf_qk_rmsnorm_rope_bwd(dq, dq_weight, dq_out, q, q_weight, dk, dk_weight, dk_out, k, k_weight, type, batch,
                           tokens, head_dim, eps, rope, workspace, workspace_bytes, stream) -> int:
    return lib().nf_qk_rmsnorm_rope_bwd(dq, dq_weight, dq_out, q, q_weight, dk, dk_weight, dk_out, k, k_weight, type,
                                        batch, tokens, head_dim, eps, rope, workspace, workspace_bytes, stream)


def nf_kv_append(k_cache, v_cache, cache_type, pages, page_size, k, v, k_weight, q_out, q, q_weight, type, tokens,
                 seqs, head_dim, starts, past, table, table_stride, max_pages, eps, rope, stream) -> int:
    return lib().nf_kv_append(k_cache, v_cache, cache_type, pages, page_size, k, v, k_weight, q_out, q, q_weight,
                              type, tokens, seqs, head_dim, starts, past, table, table_stride, max_pages, eps, rope,
                              stream)


def nf_set_path(path) -> int:
    if isinstance(path, str):
        path = PATHS[path]
    return lib().nf_set_path(path)


def nf_plan_query(op, rows, hidden) -> dict:
    if isinstance(op, str):
        op = OPS[op]
    p = Plan()
    st = lib().nf_plan_query(op, rows, hidden, ctypes.byref(p))
    if st != NF_OK:
        raise NFError(st, "nf_plan_query")
    return p.as_dict()


def nf_plan_compute(op, rows, hidden, sm_count, path=NF_PATH_AUTO):
    """Pure host planning.  Returns (status, plan dict or None)."""
    if isinstance(op, str):
        op = OPS[op]
    if isinstance(path, str):
        path = PATHS[path]
    p = Plan()
    st = lib().nf_plan_compute(op, rows, hidden, sm_count, path, ctypes.byref(p))
    return st, (p.as_dict() if st == NF_OK else None)


def nf_get_device_status(stream) -> int:
    return lib().nf_get_device_status(stream)


def nf_selftest_wait_timeout(timeout_ns, stream) -> int:
    return lib().nf_selftest_wait_timeout(timeout_ns, stream)


def nf_selftest_grid_timeout(workspace, timeout_ns, stream) -> int:
    return lib().nf_selftest_grid_timeout(workspace, timeout_ns, stream)


def nf_selftest_floor(kind, dst, src, nbytes, stream) -> int:
    return lib().nf_selftest_floor(kind, dst, src, nbytes, stream)


# ---------------------------------------------------------------- tensor helpers

def _check(st: int, where: str):
    if st != NF_OK:
        raise NFError(st, where)


def _stream(stream=None) -> int:
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _need(t, dtype, name):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _rows_hidden(x):
    hidden = x.shape[-1]
    rows = x.numel() // hidden if hidden else 0
    return rows, hidden


def _fwd_workspace(op, rows, hidden, device, workspace):
    """(pointer, bytes) of the workspace a forward call needs now: a caller
    tensor if given, else one allocated here (by PyTorch) only when the
    plan is the split or grid family."""
    import torch
    if workspace is not None:
        return workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if rows == 0 or nf_plan_query(op, rows, hidden)["path"] not in ("split", "grid"):
        return None, 0
    n = nf_workspace_size(OPS[op], rows, hidden)
    # freed right after the launch: PyTorch's allocator hands the block to
    # later work on the same stream only, which runs after these kernels
    t = torch.empty(max(n, 16), dtype=torch.uint8, device=device)
    return t.data_ptr(), n


def fused_add_rmsnorm(x, residual, weight, eps: float = 1e-6, stream=None, workspace=None):
    """In place: residual += x; x = rmsnorm(residual) * weight.  Returns (x, residual)."""
    import torch
    for t, n in ((x, "x"), (residual, "residual"), (weight, "weight")):
        _need(t, torch.bfloat16, n)
    rows, hidden = _rows_hidden(x)
    if residual.shape != x.shape or weight.shape != (hidden,):
        raise ValueError("shape mismatch")
    wp, wb = _fwd_workspace("fused_add_rmsnorm", rows, hidden, x.device, workspace)
    _check(nf_fused_add_rmsnorm_ws(x.data_ptr(), residual.data_ptr(), weight.data_ptr(), rows,
                                   hidden, eps, wp, wb, _stream(stream)), "nf_fused_add_rmsnorm_ws")
    return x, residual


def rmsnorm_fwd(x, weight, eps: float = 1e-6, out=None, stream=None, workspace=None):
    import torch
    _need(x, torch.bfloat16, "x")
    _need(weight, torch.bfloat16, "weight")
    rows, hidden = _rows_hidden(x)
    y = torch.empty_like(x) if out is None else out
    _need(y, torch.bfloat16, "out")
    wp, wb = _fwd_workspace("rmsnorm_fwd", rows, hidden, x.device, workspace)
    _check(nf_rmsnorm_fwd_ws(y.data_ptr(), x.data_ptr(), weight.data_ptr(), rows, hidden, eps,
                             wp, wb, _stream(stream)), "nf_rmsnorm_fwd_ws")
    return y


def layernorm_fwd(x, gamma, beta, eps: float = 1e-5, out=None, stream=None, workspace=None):
    """Returns (y bf16, mean fp32 [rows], rstd fp32 [rows])."""
    import torch
    for t, n in ((x, "x"), (gamma, "gamma"), (beta, "beta")):
        _need(t, torch.bfloat16, n)
    rows, hidden = _rows_hidden(x)
    y = torch.empty_like(x) if out is None else out
    mean = torch.empty(rows, dtype=torch.float32, device=x.device)
    rstd = torch.empty(rows, dtype=torch.float32, device=x.device)
    wp, wb = _fwd_workspace("layernorm_fwd", rows, hidden, x.device, workspace)
    _check(nf_layernorm_fwd_ws(y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), x.data_ptr(),
                               gamma.data_ptr(), beta.data_ptr(), rows, hidden, eps, wp, wb,
                               _stream(stream)), "nf_layernorm_fwd_ws")
    return y, mean, rstd


def layernorm_bwd(dy, x, mean, rstd, gamma, workspace=None, out=None, stream=None):
    """Returns (dx bf16, dgamma fp32, dbeta fp32).  The workspace is
    allocated here (by PyTorch) when not given; the library never allocates."""
    import torch
    for t, n in ((dy, "dy"), (x, "x"), (gamma, "gamma")):
        _need(t, torch.bfloat16, n)
    _need(mean, torch.float32, "mean")
    _need(rstd, torch.float32, "rstd")
    rows, hidden = _rows_hidden(x)
    dx = torch.empty_like(x) if out is None else out
    dgamma = torch.empty(hidden, dtype=torch.float32, device=x.device)
    dbeta = torch.empty(hidden, dtype=torch.float32, device=x.device)
    need = nf_layernorm_bwd_workspace_size(rows, hidden)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=x.device)
    _check(nf_layernorm_bwd(dx.data_ptr(), dgamma.data_ptr(), dbeta.data_ptr(), dy.data_ptr(),
                            x.data_ptr(), mean.data_ptr(), rstd.data_ptr(), gamma.data_ptr(), rows,
                            hidden, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                            _stream(stream)), "nf_layernorm_bwd")
    return dx, dgamma, dbeta


def rmsnorm_bwd(dy, x, weight, eps: float = 1e-6, workspace=None, out=None, stream=None):
    """Returns (dx bf16, dw fp32).  rstd is recomputed from x in the kernel."""
    import torch
    for t, n in ((dy, "dy"), (x, "x"), (weight, "weight")):
        _need(t, torch.bfloat16, n)
    rows, hidden = _rows_hidden(x)
    dx = torch.empty_like(x) if out is None else out
    dw = torch.empty(hidden, dtype=torch.float32, device=x.device)
    need = nf_rmsnorm_bwd_workspace_size(rows, hidden)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=x.device)
    _check(nf_rmsnorm_bwd(dx.data_ptr(), dw.data_ptr(), dy.data_ptr(), x.data_ptr(),
                          weight.data_ptr(), rows, hidden, eps, workspace.data_ptr(),
                          workspace.numel() * workspace.element_size(), _stream(stream)),
           "nf_rmsnorm_bwd")
    return dx, dw


def fused_add_rmsnorm_bwd(dy, residual, weight, dres=None, eps: float = 1e-6, workspace=None,
                         out=None, stream=None):
    """Backward of fused_add_rmsnorm given the saved residual output.
    Returns (dx bf16 -- the gradient of both x and residual --, dw fp32)."""
    import torch
    for t, n in ((dy, "dy"), (residual, "residual"), (weight, "weight")):
        _need(t, torch.bfloat16, n)
    if dres is not None:
        _need(dres, torch.bfloat16, "dres")
    rows, hidden = _rows_hidden(residual)
    dx = torch.empty_like(residual) if out is None else out
    dw = torch.empty(hidden, dtype=torch.float32, device=residual.device)
    need = nf_rmsnorm_bwd_workspace_size(rows, hidden)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=residual.device)
    _check(nf_fused_add_rmsnorm_bwd(dx.data_ptr(), dw.data_ptr(), dy.data_ptr(),
                                    None if dres is None else dres.data_ptr(),
                                    residual.data_ptr(), weight.data_ptr(), rows, hidden, eps,
                                    workspace.data_ptr(),
                                    workspace.numel() * workspace.element_size(), _stream(stream)),
           "nf_fused_add_rmsnorm_bwd")
    return dx, dw


def outer_norm_fwd(x, gamma, beta, eps: float = 1e-5, workspace=None, out=None, stream=None):
    """Per-column normalization over the rows.  Returns (y, mean [hidden], rstd [hidden])."""
    import torch
    for t, n in ((x, "x"), (gamma, "gamma"), (beta, "beta")):
        _need(t, torch.bfloat16, n)
    rows, hidden = _rows_hidden(x)
    y = torch.empty_like(x) if out is None else out
    mean = torch.empty(hidden, dtype=torch.float32, device=x.device)
    rstd = torch.empty(hidden, dtype=torch.float32, device=x.device)
    if workspace is None:
        workspace = torch.empty(max(nf_outer_norm_workspace_size(rows, hidden), 16),
                                dtype=torch.uint8, device=x.device)
    _check(nf_outer_norm_fwd(y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), x.data_ptr(),
                             gamma.data_ptr(), beta.data_ptr(), rows, hidden, eps,
                             workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                             _stream(stream)), "nf_outer_norm_fwd")
    return y, mean, rstd


def outer_norm_bwd(dy, x, mean, rstd, gamma, workspace=None, out=None, stream=None):
    """Returns (dx bf16, dgamma fp32, dbeta fp32)."""
    import torch
    for t, n in ((dy, "dy"), (x, "x"), (gamma, "gamma")):
        _need(t, torch.bfloat16, n)
    _need(mean, torch.float32, "mean")
    _need(rstd, torch.float32, "rstd")
    rows, hidden = _rows_hidden(x)
    dx = torch.empty_like(x) if out is None else out
    dgamma = torch.empty(hidden, dtype=torch.float32, device=x.device)
    dbeta = torch.empty(hidden, dtype=torch.float32, device=x.device)
    if workspace is None:
        workspace = torch.empty(max(nf_outer_norm_workspace_size(rows, hidden), 16),
                                dtype=torch.uint8, device=x.device)
    _check(nf_outer_norm_bwd(dx.data_ptr(), dgamma.data_ptr(), dbeta.data_ptr(), dy.data_ptr(),
                             x.data_ptr(), mean.data_ptr(), rstd.data_ptr(), gamma.data_ptr(),
                             rows, hidden, workspace.data_ptr(),
                             workspace.numel() * workspace.element_size(), _stream(stream)),
           "nf_outer_norm_bwd")
    return dx, dgamma, dbeta


# The helpers of the token-side operators and of those on heads: the checks, the outputs' allocation and
# the call are native (csrc/tensors.cpp), because a decode step's call takes
# 2 us on the GPU and the same steps in Python took 9 to 19 us on the host.

_native = None


def _helpers():
    """The native helpers (raises if they have not been built)."""
    global _native
    if _native is None:
        import torch  # noqa: F401  (its libraries first)
        lib()
        try:
            from . import _tensors as native
        except ImportError as e:
            raise RuntimeError("row_normalization_inner_gb300/_tensors.so cannot be loaded: build it with "
                               "`python -m row_normalization_inner_gb300.build` (no fallback exists)") from e
        _native = native
    return _native


def _result(r, where):
    """A helper's result, or NFError for the status that stands in its place."""
    if r.__class__ is int:
        raise NFError(r, where)
    return r


def _on(stream, helper, *args):
    """helper(*args) with `stream` as the current stream, which its outputs and workspaces then belong to."""
    import torch
    with torch.cuda.stream(stream):
        return helper(*args)


def rmsnorm_q8(x, weight, eps: float = 1e-6, fmt: str = "e4m3", group: int = 0, out=None,
               scale=None, stream=None):
    """RMSNorm with an 8-bit output.  Returns (q, scale): q of x's shape in
    float8_e4m3fn or int8 (fmt), scale fp32 of shape [...] (one per row) or
    [..., ceil(hidden / 128)] (group=128); q * scale stands for the
    normalized rows, which are not rounded to bf16 in between."""
    if stream is not None:
        return _on(stream, rmsnorm_q8, x, weight, eps, fmt, group, out, scale)
    return _result((_native or _helpers()).norm_q8(x, None, weight, eps, fmt, group, out, scale), "nf_rmsnorm_q8")


def fused_add_rmsnorm_q8(x, residual, weight, eps: float = 1e-6, fmt: str = "e4m3",
                         group: int = 0, out=None, scale=None, stream=None):
    """residual += x in place; returns (q, scale) of rmsnorm(residual) * weight
    as rmsnorm_q8 does (from the fp32 sums, as fused_add_rmsnorm).  x is left
    as it was."""
    if residual is None:
        raise TypeError("residual must be a tensor")
    if stream is not None:
        return _on(stream, fused_add_rmsnorm_q8, x, residual, weight, eps, fmt, group, out, scale)
    return _result((_native or _helpers()).norm_q8(x, residual, weight, eps, fmt, group, out, scale),
                   "nf_fused_add_rmsnorm_q8")


def embedding_fwd(ids, table, scale: float = 1.0, out=None, stream=None):
    """scale * table[ids], rounded to bf16: a tensor of shape [*ids.shape, hidden].
    ids int32 or int64; an id outside [0, vocab) gives a row of zeros."""
    if stream is not None:
        return _on(stream, embedding_fwd, ids, table, scale, out)
    return _result((_native or _helpers()).embedding_fwd(ids, table, scale, out), "nf_embedding_fwd")


def embedding_bwd(dy, ids, vocab: int, scale: float = 1.0, dtype=None, accumulate=None, out=None,
                  workspace=None, stream=None):
    """Gradient of embedding_fwd for its table: [vocab, hidden], fp32 or bf16
    (dtype, fp32 unless given), the rows without tokens zero; or, with
    accumulate (a gradient of that shape), that tensor with the sums added in
    place.  Equal ids are summed in fp32, in pieces in token order that are
    joined in a fixed grouping: the result is deterministic.  The workspace (nf_embedding_bwd_workspace_size bytes) is
    allocated here when not given."""
    if stream is not None:
        return _on(stream, embedding_bwd, dy, ids, vocab, scale, dtype, accumulate, out, workspace)
    return _result((_native or _helpers()).embedding_bwd(dy, ids, vocab, scale, dtype, accumulate, out, workspace),
                   "nf_embedding_bwd")


def token_logprob_fwd(logits, targets, temperature: float = 1.0, top: int = 0, stream=None):
    """Log probabilities of targets under softmax(logits / temperature).

    logits: [rows, vocab] bf16 or fp32, contiguous within a row; targets:
    [rows] int32 or int64.  Returns (logprob, entropy, stats, top_logprob,
    top_ids): fp32 [rows], [rows], [rows, 2] (the row's maximum and the
    logarithm of its sum of exponentials, for token_logprob_bwd), and the
    `top` most probable tokens, [rows, top] fp32 and int64 (None with top 0),
    equal ones by rising id.  Entries of -inf are masked; targets outside
    [0, vocab) give 0."""
    if stream is not None:
        return _on(stream, token_logprob_fwd, logits, targets, temperature, top)
    return _result((_native or _helpers()).token_logprob_fwd(logits, targets, temperature, top), "nf_token_logprob_fwd")


def token_logprob_bwd(logits, targets, stats, entropy, d_logprob, d_entropy=None,
                      temperature: float = 1.0, out=None, stream=None):
    """Gradient of token_logprob_fwd's logprob and entropy for the logits, in
    their type, given the gradients d_logprob and (optionally) d_entropy and
    the forward's stats and entropy.  out may be the logits themselves.  An
    out whose rows start as the logits' do (modulo 16 bytes) is written in
    whole vectors; the one allocated here is contiguous, so for an odd
    vocabulary in padded rows one of the same layout is up to four times as fast."""
    if stream is not None:
        return _on(stream, token_logprob_bwd, logits, targets, stats, entropy, d_logprob, d_entropy,
                   temperature, out)
    return _result((_native or _helpers()).token_logprob_bwd(logits, targets, stats, entropy, d_logprob, d_entropy,
                                                temperature, out), "nf_token_logprob_bwd")


def rope_rates(dim: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
               length: float = 8192.0, low: float = 1.0, high: float = 32.0, frequencies=None, device="cuda"):
    """What the operators on heads rotate by: an int64 tensor [dim / 2] on the
    device, each pair's share of a turn per position in units of 2^-64.

    The frequencies are base^(-2i / dim) radians per position, for contexts
    longer by `factor` than those of training scaled as `scaling` says: "plain"
    (not at all), "linear", "ntk" or "parts" (length: the context of training;
    pairs that turn `high` times or more in it keep their frequency, those that
    turn `low` times or less are slowed by the factor).  Or they are given:
    `frequencies`, [dim / 2] numbers.  Made once, on the host."""
    import torch
    if dim < 2 or dim % 2 or dim > HEAD_MAX_DIM:
        raise ValueError(f"dim must be even, 2 to {HEAD_MAX_DIM}, got {dim}")
    rates = torch.empty(dim // 2, dtype=torch.int64)
    if frequencies is not None:
        f = torch.as_tensor(frequencies, dtype=torch.float64, device="cpu").contiguous()
        if f.shape != (dim // 2,):
            raise ValueError("frequencies must be of shape [dim / 2]")
        _check(nf_rope_rates_of(rates.data_ptr(), f.data_ptr(), dim // 2), "nf_rope_rates_of")
    else:
        if scaling not in ROPE_SCALINGS:
            raise ValueError(f"scaling must be one of {', '.join(ROPE_SCALINGS)}, got {scaling!r}")
        _check(nf_rope_rates(rates.data_ptr(), dim, base, ROPE_SCALINGS[scaling], factor, length, low, high),
               "nf_rope_rates")
    return rates.to(device)


def rope_fwd(q, k, positions, rates, layout: str = "half", magnitude: float = 1.0, q_out=None, k_out=None,
             stream=None):
    """Queries and keys turned by their tokens' positions: (q_out, k_out).

    q, k: [batch, tokens, heads, head_dim] or [tokens, heads, head_dim], bf16 or
    fp32, in any order with contiguous heads (views of one projection's output
    need no copy); k may be None.  positions: int32 or int64, [batch, tokens] or
    [tokens].  rates: rope_rates' (2 * len(rates) elements of a head are
    turned, the rest left as they are).  layout: a pair is elements i and
    i + len(rates) ("half") or 2i and 2i + 1 ("interleaved").  q_out may be q.
    Outputs made here of up to 32 MB together are parts of one allocation, which
    lives as long as either of them; give q_out and k_out to hold them apart."""
    if stream is not None:
        return _on(stream, rope_fwd, q, k, positions, rates, layout, magnitude, q_out, k_out)
    return _result((_native or _helpers()).rope(q, k, positions, rates, layout, magnitude, q_out, k_out, False),
                   "nf_rope_fwd")


def rope_bwd(dq_out, dk_out, positions, rates, layout: str = "half", magnitude: float = 1.0, dq=None, dk=None,
             stream=None):
    """Gradient of rope_fwd for q and k: (dq, dk), given that of its outputs.
    dq may be dq_out; their memory as rope_fwd's outputs'."""
    if stream is not None:
        return _on(stream, rope_bwd, dq_out, dk_out, positions, rates, layout, magnitude, dq, dk)
    return _result((_native or _helpers()).rope(dq_out, dk_out, positions, rates, layout, magnitude, dq, dk, True),
                   "nf_rope_bwd")


def qk_rmsnorm_rope_fwd(q, k, q_weight, k_weight, positions=None, rates=None, eps: float = 1e-6,
                        layout: str = "half", magnitude: float = 1.0, q_out=None, k_out=None, stream=None):
    """RMSNorm of each query and key head (weights [head_dim], one for all
    heads of a kind), turned by the tokens' positions in the same pass (rates
    None: not turned).  Returns (q_out, k_out).  Tensors as for rope_fwd, the
    weights of their type; k and k_weight may be None; q_out may be q.  The
    outputs' memory as rope_fwd's."""
    if stream is not None:
        return _on(stream, qk_rmsnorm_rope_fwd, q, k, q_weight, k_weight, positions, rates, eps, layout, magnitude,
                   q_out, k_out)
    return _result((_native or _helpers()).qk_rmsnorm_rope_fwd(q, k, q_weight, k_weight, positions, rates, eps, layout,
                                                               magnitude, q_out, k_out), "nf_qk_rmsnorm_rope_fwd")


def qk_rmsnorm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, positions=None, rates=None, eps: float = 1e-6,
                        layout: str = "half", magnitude: float = 1.0, dq=None, dk=None, workspace=None,
                        stream=None):
    """Gradient of qk_rmsnorm_rope_fwd, given that of its outputs and its
    inputs: (dq, dk, dq_weight, dk_weight), the weights' in fp32.  dq may be
    dq_out or q.  The memory of dq and dk as rope_fwd's outputs', the weights'
    gradients in one allocation.  The workspace (nf_qk_rmsnorm_rope_bwd_workspace_size bytes)
    is allocated here when not given."""
    if stream is not None:
        return _on(stream, qk_rmsnorm_rope_bwd, dq_out, dk_out, q, k, q_weight, k_weight, positions, rates, eps, layout,
                   magnitude, dq, dk, workspace)
    return _result((_native or _helpers()).qk_rmsnorm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, positions,
                                                               rates, eps, layout, magnitude, dq, dk, workspace),
                   "nf_qk_rmsnorm_rope_bwd")


def kv_append(k, v, k_cache, v_cache, table, past, starts=None, rates=None, positions=None, q=None, q_weight=None,
              k_weight=None, eps: float = 1e-6, layout: str = "half", magnitude: float = 1.0, k_scale=None,
              v_scale=None, q_out=None, stream=None):
    """Appends new tokens' keys and values to a paged cache, in place; returns
    the queries, prepared in the same launch, or None without q.

    k, v (and q): [tokens, heads, head_dim], as for rope_fwd.  Caches: [pages,
    page_size, heads, head_dim] in any order with contiguous heads, of k's type,
    or float8_e4m3fn or int8 with scales k_scale, v_scale, fp32 [pages,
    page_size, heads]: q * scale stands for a row.  table: int32 [seqs,
    max_pages], each sequence's pages; past: int32 [seqs], its tokens in the
    cache before the call (negative: padding, nothing is written); starts: int32
    [seqs + 1], where its new tokens begin (None: one token per sequence).
    Tokens behind starts[seqs] are padding; a token without a page in the cache
    is not stored; what a slot holds that two tokens of a call share is not
    defined.  k (and q) are normalized where their weight is given and turned
    where rates are, by the token's place in its sequence unless
    positions [tokens] are given."""
    if stream is not None:
        return _on(stream, kv_append, k, v, k_cache, v_cache, table, past, starts, rates, positions, q, q_weight,
                   k_weight, eps, layout, magnitude, k_scale, v_scale, q_out)
    return _result((_native or _helpers()).kv_append(k, v, k_cache, v_cache, table, past, starts, rates, positions, q,
                                                     q_weight, k_weight, eps, layout, magnitude, k_scale, v_scale,
                                                     q_out), "nf_kv_append")


def set_path(path):
    _check(nf_set_path(path), "nf_set_path")


class forced_path:
    """Context manager: force a kernel family, restore AUTO on exit."""

    def __init__(self, path):
        self.path = path

    def __enter__(self):
        set_path(self.path)
        return self

    def __exit__(self, *exc):
        set_path(NF_PATH_AUTO)
