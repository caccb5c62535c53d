"""Python binding of libngram.so, the hashed n-gram embedding gather-sum for
MI355X (gfx950).

Argument marshalling only: every step of the path runs in the HIP kernels of
``csrc/ngram.hip`` behind the C ABI of ``include/ngram.h``; the functions here
check tensor dtypes and devices, pass raw pointers and the current HIP stream,
and raise on a non-zero status.  torch supplies device memory and streams.
There is no fallback: without the built library every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import NamedTuple, Optional

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libngram.so")

K = 16
PAD_ID = (1 << 21) - 1
TABLE_BF16 = 0
TABLE_INT8_ROWSCALE = 1
TABLE_MXFP4 = 2
IN_DEVICE = 0
IN_HOST = 1


class NgramError(RuntimeError):
    pass


class _Table(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row_scale", ctypes.c_void_p), ("R", ctypes.c_int64),
                ("d", ctypes.c_int32), ("dtype", ctypes.c_int32), ("location", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class _Launch(ctypes.Structure):
    _fields_ = [("tokens_per_workgroup", ctypes.c_int32), ("host_workgroups", ctypes.c_int32)]


class _Pool(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row_scale", ctypes.c_void_p), ("slot_of_row", ctypes.c_void_p),
                ("pool_rows", ctypes.c_int64), ("cached", ctypes.c_int64)]


class _Fp8(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("block_rows", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class _AdamWTensor(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("g", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("rng_offset", ctypes.c_int64), ("p_dtype", ctypes.c_int32), ("g_dtype", ctypes.c_int32),
                ("state", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class _AdamWStep(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("grad_scale", ctypes.c_double),
                ("step", ctypes.c_int64), ("seed", ctypes.c_uint64)]


class _Int4(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("zeros", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("group", ctypes.c_int32), ("scale_dtype", ctypes.c_int32)]


class _BeamState(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row_bytes", ctypes.c_int64), ("stride", ctypes.c_int64)]


class _DistillArgs(ctypes.Structure):
    _fields_ = [("logits", ctypes.c_void_p), ("teacher", ctypes.c_void_p), ("ids", ctypes.c_void_p), ("teacher_lse", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("V", ctypes.c_int64), ("ld", ctypes.c_int64), ("k", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("teacher_dtype", ctypes.c_int32), ("temperature", ctypes.c_float)]


_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_SIGNATURES = {
    "ngram_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "ngram_last_error": (ctypes.c_char_p, []),
    "ngram_version": (ctypes.c_int, []),
    "ngram_default_seeds": (None, [_P]),
    "ngram_hash": (ctypes.c_int, [_P, _I64, _P, _I32, _P, _P, _I64, _P, _P]),
    "ngram_embed_bag": (ctypes.c_int, [ctypes.POINTER(_Table), _P, _I64, _P, _P]),
    "ngram_embed_bag_ex": (ctypes.c_int, [ctypes.POINTER(_Table), _P, _I64, _P, ctypes.POINTER(_Launch), _P]),
    "ngram_gate_add": (ctypes.c_int, [_P, _P, _I64, _I32, _P, _I64, _P, _P, _P, _P]),
    "ngram_forward": (ctypes.c_int, [_P, _I64, _P, _I32, _P, _P, ctypes.POINTER(_Table), _P, _I64,
                                     _P, _P, _P, _P, _P]),
    "ngram_forward_ex": (ctypes.c_int, [_P, _I64, _P, _I32, _P, _P, ctypes.POINTER(_Table), _P, _I64,
                                        _P, _P, _P, _P, ctypes.POINTER(_Launch), _P]),
    "ngram_forward_gated": (ctypes.c_int, [_P, _I64, _P, _I32, _P, _P, ctypes.POINTER(_Table), _P, _I64,
                                           _P, _P, _P, _P, ctypes.c_float, ctypes.c_float, _P, _P, _P, _P, _P]),
    "ngram_forward_gated_ex": (ctypes.c_int, [_P, _I64, _P, _I32, _P, _P, ctypes.POINTER(_Table), _P, _I64,
                                              _P, _P, _P, _P, ctypes.c_float, ctypes.c_float, _P, _P, _P, _P,
                                              ctypes.POINTER(_Launch), _P]),
    "ngram_norm_gate_add": (ctypes.c_int, [_P, _P, _I64, _I32, _P, _I64, _P, _P, _P, _P, ctypes.c_float,
                                           ctypes.c_float, _P, _P, _P, _P]),
    "ngram_project": (ctypes.c_int, [_P, _I64, _I32, _P, _I32, _P, _P]),
    "ngram_embed_bag_bf16": (ctypes.c_int, [ctypes.POINTER(_Table), _P, _I64, _P, _P]),
    "ngram_host_alloc": (ctypes.c_int, [_I64, ctypes.POINTER(ctypes.c_void_p)]),
    "ngram_host_free": (ctypes.c_int, [_P]),
    "ngram_gather_host_workspace_bytes": (ctypes.c_int64, [_I64, _I32]),
    "ngram_gather_host_pinned_bytes": (ctypes.c_int64, [_I64]),
    "ngram_gather_host": (ctypes.c_int, [ctypes.POINTER(_Table), _P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _P,
                                         _I32, _P]),
    "ngram_pool_workspace_bytes": (ctypes.c_int64, [_I64]),
    "ngram_pool_reset": (ctypes.c_int, [ctypes.POINTER(_Table), ctypes.POINTER(_Pool), _P]),
    "ngram_pool_cache_rows": (ctypes.c_int, [ctypes.POINTER(_Table), ctypes.POINTER(_Pool), _P, _I64, _P]),
    "ngram_pool_gather": (ctypes.c_int, [ctypes.POINTER(_Table), ctypes.POINTER(_Pool), _P, _I64, _P, _P, _P,
                                         _I64, _P]),
    "ngram_count_rows": (ctypes.c_int, [_P, _I64, _I64, _P, _I32, _P]),
    "ngram_grad_workspace_bytes": (ctypes.c_int64, [_I64, _I32]),
    "ngram_grad_table": (ctypes.c_int, [_P, _I64, _I32, _I64, _P, _P, _P, _P, _P, _P, _I64, _P]),
    "ngram_grad_e1": (ctypes.c_int, [_P, _P, _I64, _I32, _I64, _P, _P, _P, _P, _P, _I64, _P]),
    "ngram_grad_gate": (ctypes.c_int, [_P, _P, _P, _I64, _I32, _P, _P, _I64, _P]),
    "ngram_grad_gate_noalloc_max_elements": (ctypes.c_int64, []),
    "ngram_grad_gate_noalloc": (ctypes.c_int, [_P, _P, _P, _I64, _I32, _P, _P]),
    "ngram_select_hot_rows": (ctypes.c_int, [_P, _I64, _I64, _P, ctypes.POINTER(ctypes.c_int64), _P, _I64, _P]),
    "ngram_fp8_code_bytes": (ctypes.c_int64, [_I64, _I64]),
    "ngram_fp8_scale_bytes": (ctypes.c_int64, [_I64, _I64, _I32]),
    "ngram_quant_fp8": (ctypes.c_int, [_P, _I32, _I64, _I32, ctypes.POINTER(_Fp8), ctypes.POINTER(_Fp8), _P]),
    "ngram_add_norm": (ctypes.c_int, [_P, _I32, _P, _I64, _I32, _P, ctypes.c_float, _P, _P, ctypes.POINTER(_Fp8), _P,
                                      _P]),
    "ngram_add_norm_grad_workspace_bytes": (ctypes.c_int64, [_I64, _I32]),
    "ngram_add_norm_grad": (ctypes.c_int, [_P, _I32, _P, _P, _P, _P, _I64, _I32, _P, _P, _P, _I64, _P]),
    "ngram_project_fp8_workspace_bytes": (ctypes.c_int64, [_I64, _I64, _I64, _I32]),
    "ngram_project_fp8": (ctypes.c_int, [ctypes.POINTER(_Fp8), ctypes.POINTER(_Fp8), _P, _I32, _P, _I64, _P]),
    "ngram_adamw": (ctypes.c_int, [ctypes.POINTER(_AdamWTensor), _I32, ctypes.POINTER(_AdamWStep), _P]),
    "ngram_adamw_rows": (ctypes.c_int, [ctypes.POINTER(_AdamWTensor), _I64, _I32, _P, _I64, _P,
                                        ctypes.POINTER(_AdamWStep), _P]),
    "ngram_int4_code_bytes": (ctypes.c_int64, [_I64, _I64]),
    "ngram_int4_scales": (ctypes.c_int64, [_I64, _I64, _I32]),
    "ngram_quant_int4": (ctypes.c_int, [_P, _I32, _I64, _I32, ctypes.POINTER(_Int4), _P]),
    "ngram_dequant_int4": (ctypes.c_int, [ctypes.POINTER(_Int4), _P, _I32, _P]),
    "ngram_project_int4": (ctypes.c_int, [_P, _I32, _I64, ctypes.POINTER(_Int4), _P, _I32, _P]),
    "ngram_beam_step_workspace_bytes": (ctypes.c_int64, [_I64, _I32, _I64, _I32]),
    "ngram_beam_step": (ctypes.c_int, [_P, _I32, _I64, _I32, _I64, _I64, _P, _P, _P, _P, _I32, _P, _P, _P, _P, _P, _P, _I64, _P]),
    "ngram_beam_reorder": (ctypes.c_int, [ctypes.POINTER(_BeamState), _I32, _P, _I64, _I32, _P]),
    "ngram_distill_workspace_bytes": (ctypes.c_int64, [_I64, _I64, _I32, _I32]),
    "ngram_distill": (ctypes.c_int, [ctypes.POINTER(_DistillArgs), _P, _P, _P, ctypes.c_float, _P, _I64, _P, _I64, _P]),
    "ngram_distill_grad": (ctypes.c_int, [ctypes.POINTER(_DistillArgs), _P, _P, ctypes.c_float, _P, _I64, _P]),
}

_lib = None


def lib():
    """The loaded libngram.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise NgramError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                             "(there is no fallback path)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(rc: int, what: str):
    if rc != 0:
        L = lib()
        raise NgramError(f"{what}: {L.ngram_status_string(rc).decode()} "
                         f"({L.ngram_last_error().decode()})")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dev(t, dtypes, name, allow_none=False):
    if t is None:
        if allow_none:
            return
        raise NgramError(f"{name} is required")
    if not t.is_cuda:
        raise NgramError(f"{name} must be a device tensor")
    if t.dtype not in dtypes:
        raise NgramError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise NgramError(f"{name} must be contiguous")


def _need(t, count, name):
    """Refuse a buffer smaller than the call reads or writes."""
    if t is not None and t.numel() < count:
        raise NgramError(f"{name} holds {t.numel()} elements, the call needs {count}")


_BF16 = (torch.bfloat16, torch.int16, torch.uint16)
_I32T = (torch.int32,)
_F32 = (torch.float32,)


def default_seeds():
    s = (ctypes.c_uint64 * K)()
    lib().ngram_default_seeds(s)
    return [int(x) for x in s]


def _launch_arg(launch):
    """``launch``: None, or (tokens_per_workgroup, host_workgroups), 0 for the
    library's choice of either."""
    if launch is None:
        return None
    tpw, hw = launch
    return ctypes.byref(_Launch(int(tpw), int(hw)))


def _seeds_arg(seeds):
    if seeds is None:
        return None
    if len(seeds) != K:
        raise NgramError("seeds must hold 16 values")
    return (ctypes.c_uint64 * K)(*[int(s) & 0xFFFFFFFFFFFFFFFF for s in seeds])


class Table:
    """An n-gram table: ``data`` [R][d] bf16 (or int8 with ``row_scale`` [R]
    fp32) in device memory, or a ``HostBuffer`` in pinned host memory."""

    def __init__(self, data, R: int, d: int, dtype: int = TABLE_BF16, row_scale=None):
        self.data = data
        self.row_scale = row_scale
        self.R, self.d, self.dtype = int(R), int(d), int(dtype)
        nbytes = self.R * row_bytes(self.d, self.dtype)
        if isinstance(data, HostBuffer):
            self.location = IN_HOST
            ptr = data.ptr
            if data.nbytes < nbytes:
                raise NgramError("host table buffer is smaller than R rows")
        else:
            dts = {TABLE_BF16: _BF16, TABLE_INT8_ROWSCALE: (torch.int8,), TABLE_MXFP4: (torch.uint8, torch.int8)}
            _dev(data, dts.get(self.dtype, _BF16), "table")
            if data.numel() * data.element_size() < nbytes:
                raise NgramError(f"table holds {data.numel() * data.element_size()} bytes, R rows need {nbytes}")
            self.location = IN_DEVICE
            ptr = data.data_ptr()
        if dtype == TABLE_INT8_ROWSCALE:
            _dev(row_scale, _F32, "row_scale")
            _need(row_scale, self.R, "row_scale")
        self._c = _Table(ptr, None if row_scale is None else row_scale.data_ptr(), self.R, self.d,
                         self.dtype, self.location, 0)

    @property
    def c(self):
        return ctypes.byref(self._c)


class HostBuffer:
    """Pinned, device-mapped host memory from ngram_host_alloc."""

    def __init__(self, nbytes: int):
        p = ctypes.c_void_p()
        _check(lib().ngram_host_alloc(int(nbytes), ctypes.byref(p)), "ngram_host_alloc")
        self.ptr = p.value
        self.nbytes = int(nbytes)

    def numpy(self, dtype, shape):
        import numpy as np
        buf = (ctypes.c_char * self.nbytes).from_address(self.ptr)
        return np.frombuffer(buf, dtype=dtype, count=int(np.prod(shape))).reshape(shape)

    def free(self):
        if self.ptr:
            _check(lib().ngram_host_free(ctypes.c_void_p(self.ptr)), "ngram_host_free")
            self.ptr = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def row_bytes(d: int, dtype: int) -> int:
    """Bytes of one table row: 2d (bf16), d (int8) or d/2 + d/32 (MXFP4)."""
    if dtype == TABLE_BF16:
        return 2 * d
    if dtype == TABLE_MXFP4:
        return d // 2 + d // 32
    return d


def _vocab(e1, d):
    """Rows of the [V][d] e1 table (any shape with V*d elements)."""
    if e1 is None:
        return 0
    if e1.numel() % d:
        raise NgramError(f"e1 has {e1.numel()} elements, not a multiple of d={d}")
    return e1.numel() // d


def ngram_hash(tokens, seq_offsets, R, rows_out=None, history=None, seeds=None, stream=None):
    _dev(tokens, _I32T, "tokens")
    _dev(seq_offsets, _I32T, "seq_offsets")
    _dev(history, _I32T, "history", allow_none=True)
    n = tokens.numel()
    if rows_out is None:
        rows_out = torch.empty((n, K), dtype=torch.int32, device=tokens.device)
    _dev(rows_out, _I32T, "rows_out")
    _need(rows_out, n * K, "rows_out")
    _need(history, 2 * (seq_offsets.numel() - 1), "history")
    _check(lib().ngram_hash(_ptr(tokens), n, _ptr(seq_offsets), seq_offsets.numel() - 1,
                            _ptr(history), _seeds_arg(seeds), int(R), _ptr(rows_out), _stream(stream)),
           "ngram_hash")
    return rows_out


def ngram_embed_bag(table: Table, rows, eN_out=None, launch=None, stream=None):
    _dev(rows, _I32T, "rows")
    n = rows.shape[0] if rows.dim() == 2 else rows.numel() // K
    if eN_out is None:
        eN_out = torch.empty((n, table.d), dtype=torch.float32, device=rows.device)
    _dev(eN_out, _F32, "eN_out")
    _need(rows, n * K, "rows")
    _need(eN_out, n * table.d, "eN_out")
    if launch is None:
        rc = lib().ngram_embed_bag(table.c, _ptr(rows), n, _ptr(eN_out), _stream(stream))
    else:
        rc = lib().ngram_embed_bag_ex(table.c, _ptr(rows), n, _ptr(eN_out), _launch_arg(launch), _stream(stream))
    _check(rc, "ngram_embed_bag")
    return eN_out


def ngram_gate_add(eN, tokens, W_g, out, e1=None, residual=None, stream=None):
    _dev(eN, _F32, "eN")
    _dev(tokens, _I32T, "tokens")
    _dev(W_g, _F32, "W_g")
    _dev(out, _BF16, "out")
    _dev(e1, _BF16, "e1", allow_none=True)
    _dev(residual, _BF16, "residual", allow_none=True)
    n, d = eN.shape
    V = _vocab(e1, d)
    _need(tokens, n, "tokens")
    _need(W_g, d, "W_g")
    _need(out, n * d, "out")
    _need(residual, n * d, "residual")
    _check(lib().ngram_gate_add(_ptr(eN), _ptr(tokens), n, d, _ptr(e1), V, _ptr(W_g),
                                _ptr(residual), _ptr(out), _stream(stream)), "ngram_gate_add")
    return out


def ngram_forward(tokens, seq_offsets, table: Table, W_g, out, e1=None, residual=None,
                  history=None, seeds=None, rows_out=None, launch=None, stream=None):
    _dev(tokens, _I32T, "tokens")
    _dev(seq_offsets, _I32T, "seq_offsets")
    _dev(history, _I32T, "history", allow_none=True)
    _dev(W_g, _F32, "W_g")
    _dev(out, _BF16, "out")
    _dev(e1, _BF16, "e1", allow_none=True)
    _dev(residual, _BF16, "residual", allow_none=True)
    _dev(rows_out, _I32T, "rows_out", allow_none=True)
    V = _vocab(e1, table.d)
    n, d = tokens.numel(), table.d
    _need(W_g, d, "W_g")
    _need(out, n * d, "out")
    _need(residual, n * d, "residual")
    _need(rows_out, n * K, "rows_out")
    _need(history, 2 * (seq_offsets.numel() - 1), "history")
    args = (_ptr(tokens), tokens.numel(), _ptr(seq_offsets), seq_offsets.numel() - 1, _ptr(history),
            _seeds_arg(seeds), table.c, _ptr(e1), V, _ptr(W_g), _ptr(residual), _ptr(out), _ptr(rows_out))
    if launch is None:
        rc = lib().ngram_forward(*args, _stream(stream))
    else:
        rc = lib().ngram_forward_ex(*args, _launch_arg(launch), _stream(stream))
    _check(rc, "ngram_forward")
    return out


def ngram_forward_gated(tokens, seq_offsets, table: Table, W_g, gamma, u, v, b, eps, out, e1,
                        residual=None, history=None, seeds=None, rows_out=None, stats_out=None, launch=None,
                        stream=None):
    """Normalised, input-gated forward (see ngram_forward_gated in ngram.h);
    ``stats_out`` [n][2] float64 receives (r, logit) per token."""
    _dev(tokens, _I32T, "tokens")
    _dev(seq_offsets, _I32T, "seq_offsets")
    _dev(history, _I32T, "history", allow_none=True)
    for t, name in ((W_g, "W_g"), (gamma, "gamma"), (u, "u"), (v, "v")):
        _dev(t, _F32, name)
    _dev(out, _BF16, "out")
    _dev(e1, _BF16, "e1")
    _dev(residual, _BF16, "residual", allow_none=True)
    _dev(rows_out, _I32T, "rows_out", allow_none=True)
    _dev(stats_out, (torch.float64,), "stats_out", allow_none=True)
    V = _vocab(e1, table.d)
    n, d = tokens.numel(), table.d
    for t, name in ((W_g, "W_g"), (gamma, "gamma"), (u, "u"), (v, "v")):
        _need(t, d, name)
    _need(out, n * d, "out")
    _need(residual, n * d, "residual")
    _need(rows_out, n * K, "rows_out")
    _need(stats_out, 2 * n, "stats_out")
    _need(history, 2 * (seq_offsets.numel() - 1), "history")
    args = (_ptr(tokens), n, _ptr(seq_offsets), seq_offsets.numel() - 1, _ptr(history), _seeds_arg(seeds),
            table.c, _ptr(e1), V, _ptr(W_g), _ptr(gamma), _ptr(u), _ptr(v), float(b), float(eps), _ptr(residual),
            _ptr(out), _ptr(rows_out), _ptr(stats_out))
    if launch is None:
        rc = lib().ngram_forward_gated(*args, _stream(stream))
    else:
        rc = lib().ngram_forward_gated_ex(*args, _launch_arg(launch), _stream(stream))
    _check(rc, "ngram_forward_gated")
    return out


def ngram_norm_gate_add(eN, tokens, e1, W_g, gamma, u, v, b, eps, out, residual=None, stats_out=None,
                        stream=None):
    """The normalised, input-gated epilogue on given fp32 sums eN [n][d]
    (see ngram_norm_gate_add in ngram.h)."""
    _dev(eN, _F32, "eN")
    _dev(tokens, _I32T, "tokens")
    for t, name in ((W_g, "W_g"), (gamma, "gamma"), (u, "u"), (v, "v")):
        _dev(t, _F32, name)
    _dev(out, _BF16, "out")
    _dev(e1, _BF16, "e1")
    _dev(residual, _BF16, "residual", allow_none=True)
    _dev(stats_out, (torch.float64,), "stats_out", allow_none=True)
    n, d = eN.shape
    V = _vocab(e1, d)
    _need(tokens, n, "tokens")
    for t, name in ((W_g, "W_g"), (gamma, "gamma"), (u, "u"), (v, "v")):
        _need(t, d, name)
    _need(out, n * d, "out")
    _need(residual, n * d, "residual")
    _need(stats_out, 2 * n, "stats_out")
    _check(lib().ngram_norm_gate_add(_ptr(eN), _ptr(tokens), n, d, _ptr(e1), V, _ptr(W_g), _ptr(gamma), _ptr(u),
                                     _ptr(v), float(b), float(eps), _ptr(residual), _ptr(out), _ptr(stats_out),
                                     _stream(stream)), "ngram_norm_gate_add")
    return out


def ngram_embed_bag_bf16(table: Table, rows, out=None, stream=None):
    """The sums of ngram_embed_bag rounded to bf16: out [n][d] (bf16 bits)."""
    _dev(rows, _I32T, "rows")
    n = rows.shape[0]
    if out is None:
        out = torch.empty((n, table.d), dtype=torch.int16, device=rows.device)
    _dev(out, _BF16, "out")
    _need(out, n * table.d, "out")
    _check(lib().ngram_embed_bag_bf16(table.c, _ptr(rows), n, _ptr(out), _stream(stream)), "ngram_embed_bag_bf16")
    return out


def ngram_project(x, P, y=None, stream=None):
    """y [n][d_out] fp32 = P x for x [n][d_in] and P [d_out][d_in], both bf16
    bits (int16 tensors); see ngram_project in ngram.h."""
    _dev(x, _BF16, "x")
    _dev(P, _BF16, "P")
    n, d_in = x.shape
    d_out = P.shape[0]
    if P.dim() != 2 or P.shape[1] != d_in:
        raise NgramError(f"P must be [d_out][{d_in}], got {tuple(P.shape)}")
    if y is None:
        y = torch.empty((n, d_out), dtype=torch.float32, device=x.device)
    _dev(y, _F32, "y")
    _need(y, n * d_out, "y")
    _check(lib().ngram_project(_ptr(x), n, d_in, _ptr(P), d_out, _ptr(y), _stream(stream)), "ngram_project")
    return y


GATHER_ZERO_COPY = 0
GATHER_ASYNC_COPY = 1


def gather_host_workspace(n: int, d: int, device="cuda:0"):
    nbytes = int(lib().ngram_gather_host_workspace_bytes(int(n), int(d)))
    return torch.empty((nbytes + 15) // 16 * 16, dtype=torch.uint8, device=device)


def gather_host_pinned(n: int) -> "HostBuffer":
    """Pinned host memory for ngram_gather_host's async-copy mode."""
    return HostBuffer(max(16, int(lib().ngram_gather_host_pinned_bytes(int(n)))))


def ngram_gather_host(table: Table, rows, stage_out, remap_out, stage_scale_out=None, n_staged_out=None,
                      mode=GATHER_ZERO_COPY, workspace=None, pinned=None, stream=None):
    """Stage the batch's distinct rows of a pinned-host table in device
    memory.  Returns (stage_out, remap_out, n_staged_out [1] int64)."""
    _dev(rows, _I32T, "rows")
    _dev(remap_out, _I32T, "remap_out")
    _dev(stage_scale_out, _F32, "stage_scale_out", allow_none=True)
    if not stage_out.is_cuda or not stage_out.is_contiguous():
        raise NgramError("stage_out must be a contiguous device tensor")
    n = rows.shape[0] if rows.dim() == 2 else rows.numel() // K
    _need(rows, n * K, "rows")
    _need(remap_out, n * K, "remap_out")
    rb = row_bytes(table.d, table.dtype)
    if stage_out.numel() * stage_out.element_size() < n * K * rb:
        raise NgramError("stage_out is smaller than n * 16 rows")
    if table.dtype == TABLE_INT8_ROWSCALE:
        _need(stage_scale_out, n * K, "stage_scale_out")
    if n_staged_out is None:
        n_staged_out = torch.empty(1, dtype=torch.int64, device=rows.device)
    _dev(n_staged_out, (torch.int64,), "n_staged_out")
    if workspace is None:
        workspace = gather_host_workspace(n, table.d, rows.device)
    own_pinned = None
    if mode == GATHER_ASYNC_COPY and pinned is None:
        own_pinned = pinned = gather_host_pinned(n)
    p_ptr = None if pinned is None else ctypes.c_void_p(pinned.ptr)
    p_bytes = 0 if pinned is None else pinned.nbytes
    _check(lib().ngram_gather_host(table.c, _ptr(rows), n, _ptr(workspace), workspace.numel() * workspace.element_size(),
                                   p_ptr, p_bytes, _ptr(stage_out), _ptr(stage_scale_out), _ptr(remap_out),
                                   _ptr(n_staged_out), int(mode), _stream(stream)), "ngram_gather_host")
    if own_pinned is not None:
        # the copies read only the table, but the row list they were built
        # from sits in this buffer: let the stream pass them before freeing it
        (stream or torch.cuda.current_stream()).synchronize()
        own_pinned.free()
    return stage_out, remap_out, n_staged_out


class RowPool:
    """Device-memory row pool in front of a pinned-host table: ``pool_rows``
    rows of the table's dtype (a hot-row cache in the first ``cached`` rows,
    staged misses after them), per-row scales for int8, and the [R] map
    ``slot_of_row``.  The buffers are torch device tensors."""

    def __init__(self, table: Table, pool_rows: int, device="cuda:0", stream=None):
        if table.location != IN_HOST:
            raise NgramError("a row pool fronts a table in host memory")
        self.table = table
        self.pool_rows = int(pool_rows)
        if table.dtype == TABLE_MXFP4:
            self.data = torch.empty(self.pool_rows * row_bytes(table.d, table.dtype), dtype=torch.uint8,
                                    device=device)
        else:
            dt = torch.int16 if table.dtype == TABLE_BF16 else torch.int8
            self.data = torch.empty(self.pool_rows * table.d, dtype=dt, device=device)
        self.row_scale = (torch.empty(self.pool_rows, dtype=torch.float32, device=device)
                          if table.dtype == TABLE_INT8_ROWSCALE else None)
        self.slot_of_row = torch.empty(table.R, dtype=torch.int32, device=device)
        self._c = _Pool(self.data.data_ptr(), None if self.row_scale is None else self.row_scale.data_ptr(),
                        self.slot_of_row.data_ptr(), self.pool_rows, 0)
        _check(lib().ngram_pool_reset(table.c, ctypes.byref(self._c), _stream(stream)), "ngram_pool_reset")

    @property
    def cached(self):
        return int(self._c.cached)

    def device_table(self) -> Table:
        """The pool as a device table of ``pool_rows`` rows."""
        return Table(self.data, self.pool_rows, self.table.d, self.table.dtype, row_scale=self.row_scale)


def ngram_pool_workspace_bytes(n: int) -> int:
    return int(lib().ngram_pool_workspace_bytes(int(n)))


def pool_workspace(n: int, device="cuda:0"):
    nbytes = ngram_pool_workspace_bytes(n)
    return torch.empty((nbytes + 15) // 16 * 16, dtype=torch.uint8, device=device)


def ngram_pool_reset(pool: RowPool, stream=None):
    _check(lib().ngram_pool_reset(pool.table.c, ctypes.byref(pool._c), _stream(stream)), "ngram_pool_reset")


def ngram_pool_cache_rows(pool: RowPool, hot_rows, C=None, stream=None):
    _dev(hot_rows, _I32T, "hot_rows")
    C = hot_rows.numel() if C is None else int(C)
    _need(hot_rows, C, "hot_rows")
    _check(lib().ngram_pool_cache_rows(pool.table.c, ctypes.byref(pool._c), _ptr(hot_rows), C, _stream(stream)),
           "ngram_pool_cache_rows")


def ngram_pool_gather(pool: RowPool, rows, pool_rows_out=None, fetched_out=None, workspace=None, stream=None):
    _dev(rows, _I32T, "rows")
    n = rows.shape[0] if rows.dim() == 2 else rows.numel() // K
    _need(rows, n * K, "rows")
    if pool_rows_out is None:
        pool_rows_out = torch.empty((n, K), dtype=torch.int32, device=rows.device)
    _dev(pool_rows_out, _I32T, "pool_rows_out")
    _need(pool_rows_out, n * K, "pool_rows_out")
    if fetched_out is not None:
        _dev(fetched_out, (torch.int64,), "fetched_out")
    if workspace is None:
        workspace = pool_workspace(n, rows.device)
    _check(lib().ngram_pool_gather(pool.table.c, ctypes.byref(pool._c), _ptr(rows), n, _ptr(pool_rows_out),
                                   _ptr(fetched_out), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                   _stream(stream)), "ngram_pool_gather")
    return pool_rows_out


def ngram_count_rows(rows, R, counts=None, accumulate=False, stream=None):
    _dev(rows, _I32T, "rows")
    n = rows.shape[0] if rows.dim() == 2 else rows.numel() // K
    if counts is None:
        counts = torch.empty(int(R), dtype=torch.int32, device=rows.device)
        accumulate = False
    _dev(counts, _I32T, "counts")
    _need(counts, int(R), "counts")
    _check(lib().ngram_count_rows(_ptr(rows), n, int(R), _ptr(counts), 1 if accumulate else 0, _stream(stream)),
           "ngram_count_rows")
    return counts


def ngram_select_hot_rows(counts, C, hot_rows_out=None, workspace=None, stream=None):
    """Returns (hot_rows_out, selected); synchronizes the stream."""
    _dev(counts, _I32T, "counts")
    if hot_rows_out is None:
        hot_rows_out = torch.empty(max(int(C), 1), dtype=torch.int32, device=counts.device)
    _dev(hot_rows_out, _I32T, "hot_rows_out")
    _need(hot_rows_out, int(C), "hot_rows_out")
    if workspace is None:
        workspace = pool_workspace(0, counts.device)
    sel = ctypes.c_int64(0)
    _check(lib().ngram_select_hot_rows(_ptr(counts), counts.numel(), int(C), _ptr(hot_rows_out), ctypes.byref(sel),
                                       _ptr(workspace), workspace.numel() * workspace.element_size(),
                                       _stream(stream)), "ngram_select_hot_rows")
    return hot_rows_out, int(sel.value)


def grad_workspace(n: int, d: int, device="cuda:0"):
    nbytes = int(lib().ngram_grad_workspace_bytes(int(n), int(d)))
    # torch's caching allocator returns 512-byte aligned blocks
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _ws_args(workspace):
    return _ptr(workspace), workspace.numel() * workspace.element_size()


def ngram_grad_table(rows, W_g, dout, R, grad_rows_out=None, grad_out=None, n_unique_out=None,
                     workspace=None, stream=None):
    """Sparse table gradient: (grad_rows_out [16n], grad_out [16n][d], n_unique_out [1] int64);
    the first n_unique_out rows are valid."""
    _dev(rows, _I32T, "rows")
    _dev(W_g, _F32, "W_g")
    _dev(dout, _BF16, "dout")
    n = rows.shape[0] if rows.dim() == 2 else rows.numel() // K
    d = dout.numel() // max(n, 1) if n else W_g.numel()
    _need(rows, n * K, "rows")
    _need(W_g, d, "W_g")
    dev = rows.device
    grad_rows_out = torch.empty(n * K, dtype=torch.int32, device=dev) if grad_rows_out is None else grad_rows_out
    grad_out = torch.empty((n * K, d), dtype=torch.float32, device=dev) if grad_out is None else grad_out
    n_unique_out = torch.empty(1, dtype=torch.int64, device=dev) if n_unique_out is None else n_unique_out
    _dev(grad_rows_out, _I32T, "grad_rows_out")
    _dev(grad_out, _F32, "grad_out")
    _dev(n_unique_out, (torch.int64,), "n_unique_out")
    _need(grad_rows_out, n * K, "grad_rows_out")
    _need(grad_out, n * K * d, "grad_out")
    workspace = grad_workspace(n, d, dev) if workspace is None else workspace
    _check(lib().ngram_grad_table(_ptr(rows), n, d, int(R), _ptr(W_g), _ptr(dout), _ptr(grad_rows_out),
                                  _ptr(grad_out), _ptr(n_unique_out), *_ws_args(workspace), _stream(stream)),
           "ngram_grad_table")
    return grad_rows_out, grad_out, n_unique_out


def ngram_grad_e1(tokens, rows, dout, V, grad_tokens_out=None, grad_out=None, n_unique_out=None,
                  workspace=None, stream=None):
    _dev(tokens, _I32T, "tokens")
    _dev(rows, _I32T, "rows")
    _dev(dout, _BF16, "dout")
    n = tokens.numel()
    d = dout.numel() // max(n, 1)
    _need(rows, n * K, "rows")
    dev = tokens.device
    grad_tokens_out = torch.empty(n, dtype=torch.int32, device=dev) if grad_tokens_out is None else grad_tokens_out
    grad_out = torch.empty((n, d), dtype=torch.float32, device=dev) if grad_out is None else grad_out
    n_unique_out = torch.empty(1, dtype=torch.int64, device=dev) if n_unique_out is None else n_unique_out
    _need(grad_tokens_out, n, "grad_tokens_out")
    _need(grad_out, n * d, "grad_out")
    workspace = grad_workspace(n, d, dev) if workspace is None else workspace
    _check(lib().ngram_grad_e1(_ptr(tokens), _ptr(rows), n, d, int(V), _ptr(dout), _ptr(grad_tokens_out),
                               _ptr(grad_out), _ptr(n_unique_out), *_ws_args(workspace), _stream(stream)),
           "ngram_grad_e1")
    return grad_tokens_out, grad_out, n_unique_out


def ngram_grad_gate(rows, dout, eN, grad_Wg_out=None, workspace=None, stream=None):
    _dev(rows, _I32T, "rows")
    _dev(dout, _BF16, "dout")
    _dev(eN, _F32, "eN")
    n, d = eN.shape
    _need(rows, n * K, "rows")
    _need(dout, n * d, "dout")
    grad_Wg_out = torch.empty(d, dtype=torch.float32, device=eN.device) if grad_Wg_out is None else grad_Wg_out
    _need(grad_Wg_out, d, "grad_Wg_out")
    workspace = grad_workspace(n, d, eN.device) if workspace is None else workspace
    _check(lib().ngram_grad_gate(_ptr(rows), _ptr(dout), _ptr(eN), n, d, _ptr(grad_Wg_out), *_ws_args(workspace),
                                 _stream(stream)), "ngram_grad_gate")
    return grad_Wg_out


def ngram_grad_gate_noalloc(rows, dout, eN, grad_Wg_out=None, stream=None):
    """The gate gradient without a workspace (the library's static scratch;
    calls that overlap on one GPU race)."""
    _dev(rows, _I32T, "rows")
    _dev(dout, _BF16, "dout")
    _dev(eN, _F32, "eN")
    n, d = eN.shape
    _need(rows, n * K, "rows")
    _need(dout, n * d, "dout")
    grad_Wg_out = torch.empty(d, dtype=torch.float32, device=eN.device) if grad_Wg_out is None else grad_Wg_out
    _dev(grad_Wg_out, _F32, "grad_Wg_out")
    _need(grad_Wg_out, d, "grad_Wg_out")
    _check(lib().ngram_grad_gate_noalloc(_ptr(rows), _ptr(dout), _ptr(eN), n, d, _ptr(grad_Wg_out), _stream(stream)),
           "ngram_grad_gate_noalloc")
    return grad_Wg_out


F32 = 0
BF16 = 1
STATE_F32 = 0
STATE_FP8 = 1
FP8_BLOCK = 128
FP8_MAX = 1 << 30

_CODES = (torch.float8_e4m3fn, torch.uint8)
_BYTES = (torch.uint8, torch.float8_e8m0fnu)
_VALUES = (torch.float32,) + _BF16

# The calls below are short on the GPU at decode sizes (a few microseconds), so
# their marshalling is kept short too: tensors go through one check each, and
# raw pointers, as ints, straight to ctypes.
#
# ``stream``: where the call's kernels run, by default the current stream.  Its
# arguments have to be ready there, and the caller lets the current stream wait
# for it before reading the results there.


def _arg(t, dtypes, count, name):
    """The pointer of a required contiguous device tensor of at least
    ``count`` elements."""
    if t is None or t.dtype not in dtypes or not t.is_cuda or not t.is_contiguous() or t.numel() < count:
        _dev(t, dtypes, name)
        _need(t, count, name)
    return t.data_ptr()


def _opt(t, dtypes, count, name):
    """The same for an optional one: None stays None."""
    return None if t is None else _arg(t, dtypes, count, name)


def _raw_stream(stream):
    """The HIP stream handle of ``stream``, by default the current device's
    current stream."""
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()) if stream is None else stream.cuda_stream


def _new(rows, cols, dtype, device, stream):
    """A contiguous [rows][cols] tensor ([rows] where cols is None) that a
    call makes for itself or for its caller; with its strides given, making it
    takes three quarters of the time.  For a given ``stream`` it is memory of
    that stream: a block of the current one's may still be in use by what is
    queued there, which the given stream does not wait for.  The allocator is
    told of the current stream, on which the caller reads it."""
    shape, strides = ((rows,), (1,)) if cols is None else ((rows, cols), (cols, 1))
    if stream is None:
        return torch.empty_strided(shape, strides, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty_strided(shape, strides, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream())
    return t


def _scratch(t):
    """(pointer, bytes) of a workspace: any contiguous device tensor."""
    if not t.is_cuda or not t.is_contiguous():
        raise NgramError("workspace must be a contiguous device tensor")
    return t.data_ptr(), t.numel() * t.element_size()


def _value(t):
    """The ngram_value of a tensor that has been checked against _VALUES."""
    return F32 if t.dtype is torch.float32 else BF16


def _matrix(t, name):
    """(rows, columns) of a matrix argument."""
    if t is None or t.dim() != 2:
        raise NgramError(f"{name} must have two dimensions")
    return t.shape


class Fp8:
    """An 8-bit matrix: E4M3 ``codes`` [rows][128 ceil(cols / 128)] and E8M0
    ``scales``, one byte per 128 columns of a row (``block_rows`` 1) or of 128
    rows (128); see "8-bit matrices" in ngram.h."""

    __slots__ = ("codes", "scales", "rows", "cols", "block_rows", "c")

    def __init__(self, codes, scales, rows: int, cols: int, block_rows: int = 1):
        ld, srows, sld = _fp8_shape(rows, cols, block_rows)
        self.rows, self.cols, self.block_rows = rows, cols, block_rows
        self.codes, self.scales = codes, scales
        self.c = _Fp8(_arg(codes, _CODES, rows * ld, "codes"), _arg(scales, _BYTES, srows * sld, "scales"), rows, cols, block_rows, 0)

    @classmethod
    def empty(cls, rows: int, cols: int, block_rows: int = 1, device="cuda:0", stream=None) -> "Fp8":
        if torch.device(device).type != "cuda":
            raise NgramError(f"an 8-bit matrix lies on a GPU, not on device {device}")
        return cls._empty(rows, cols, block_rows, device, stream)

    @classmethod
    def _empty(cls, rows, cols, block_rows, device, stream):
        ld, srows, sld = _fp8_shape(rows, cols, block_rows)
        codes = _new(rows, ld, torch.float8_e4m3fn, device, stream)
        scales = _new(srows, sld, torch.uint8, device, stream)
        self = cls.__new__(cls)
        self.rows, self.cols, self.block_rows, self.codes, self.scales = rows, cols, block_rows, codes, scales
        self.c = _Fp8(codes.data_ptr(), scales.data_ptr(), rows, cols, block_rows, 0)
        return self


def _fp8_shape(rows, cols, block_rows):
    """(code bytes a row, scale rows, scale bytes a row), as
    ngram_fp8_code_bytes and ngram_fp8_scale_bytes count them."""
    if not (0 <= rows <= FP8_MAX and 0 <= cols <= FP8_MAX) or block_rows not in (1, FP8_BLOCK):
        raise NgramError(f"no 8-bit matrix has rows={rows}, cols={cols}, block_rows={block_rows}")
    nb = (cols + FP8_BLOCK - 1) // FP8_BLOCK
    return nb * FP8_BLOCK, rows if block_rows == 1 else (rows + FP8_BLOCK - 1) // FP8_BLOCK, (nb + 3) // 4 * 4


def _fp8_c(q):
    return None if q is None else q.c


def ngram_quant_fp8(x, rows=True, transposed=False, block_rows: int = 1, q=None, qt=None, stream=None):
    """x [n][d] (fp32 or bf16) in 8 bits: (q, qt), with None for the one that
    is not wanted.  ``rows``: q, n x d; ``transposed``: qt, d x n; or pass
    the Fp8 to fill.  See ngram_quant_fp8 in ngram.h."""
    n, d = _matrix(x, "x")
    px = _arg(x, _VALUES, n * d, "x")
    if q is None and rows:
        q = Fp8._empty(n, d, block_rows, x.device, stream)
    if qt is None and transposed:
        qt = Fp8._empty(d, n, block_rows, x.device, stream)
    rc = lib().ngram_quant_fp8(px, _value(x), n, d, _fp8_c(q), _fp8_c(qt), _raw_stream(stream))
    if rc:
        _check(rc, "ngram_quant_fp8")
    return q, qt


class NormOut(NamedTuple):
    """ngram_add_norm's outputs; None for those not asked for."""
    sum: Optional[torch.Tensor]
    y: Optional[torch.Tensor]
    q: Optional[Fp8]
    r: Optional[torch.Tensor]


def ngram_add_norm(x, gamma, eps, residual=None, sum_out=None, y_out=None, q_out=None, r_out=None, quantise=True,
                   keep_y=False, keep_r=False, stream=None) -> NormOut:
    """s = bf16(residual + x), y = s / rms(s) * gamma, and y in 8 bits, in one
    pass (see ngram_add_norm in ngram.h).  ``sum_out`` receives s and may be
    ``residual``; q, y (bf16) and r = 1 / rms are made where ``quantise``,
    ``keep_y`` and ``keep_r`` ask for them or a buffer is passed."""
    n, d = _matrix(x, "x")
    count = n * d
    px = _arg(x, _VALUES, count, "x")
    pg = _arg(gamma, _F32, d, "gamma")
    if q_out is None and quantise:
        q_out = Fp8._empty(n, d, 1, x.device, stream)
    if y_out is None and keep_y:
        y_out = _new(n, d, torch.bfloat16, x.device, stream)
    if r_out is None and keep_r:
        r_out = _new(n, None, torch.float32, x.device, stream)
    rc = lib().ngram_add_norm(px, _value(x), _opt(residual, _BF16, count, "residual"), n, d, pg, eps,
                              _opt(sum_out, _BF16, count, "sum_out"), _opt(y_out, _BF16, count, "y_out"), _fp8_c(q_out),
                              _opt(r_out, _F32, n, "r_out"), _raw_stream(stream))
    if rc:
        _check(rc, "ngram_add_norm")
    return NormOut(sum_out, y_out, q_out, r_out)


def add_norm_grad_workspace(n: int, d: int, device="cuda:0", stream=None):
    """Workspace of ngram_add_norm_grad, on ``stream`` (by default the current one)."""
    nbytes = lib().ngram_add_norm_grad_workspace_bytes(n, d)
    if nbytes < 0:
        raise NgramError(f"no norm gradient has n={n}, d={d}")
    return _new(nbytes, None, torch.uint8, device, stream)


def ngram_add_norm_grad(dy, sum, r, gamma, dsum=None, dx_out=None, dgamma_out=None, workspace=None, stream=None):
    """(dx [n][d] bf16, dgamma [d] fp32) from dL/dy (fp32 or bf16) and the
    forward's sum and r; ``dsum`` is the gradient that reaches the sum along
    the residual stream (see ngram_add_norm_grad in ngram.h)."""
    n, d = _matrix(dy, "dy")
    count = n * d
    pdy = _arg(dy, _VALUES, count, "dy")
    ps, pr, pg = _arg(sum, _BF16, count, "sum"), _arg(r, _F32, n, "r"), _arg(gamma, _F32, d, "gamma")
    if dx_out is None:
        dx_out = _new(n, d, torch.bfloat16, dy.device, stream)
    if dgamma_out is None:
        dgamma_out = _new(d, None, torch.float32, dy.device, stream)
    if workspace is None:
        workspace = add_norm_grad_workspace(n, d, dy.device, stream)
    ws, ws_bytes = _scratch(workspace)
    rc = lib().ngram_add_norm_grad(pdy, _value(dy), ps, pr, pg, _opt(dsum, _BF16, count, "dsum"), n, d,
                                   _arg(dx_out, _BF16, count, "dx_out"), _arg(dgamma_out, _F32, d, "dgamma_out"),
                                   ws, ws_bytes, _raw_stream(stream))
    if rc:
        _check(rc, "ngram_add_norm_grad")
    return dx_out, dgamma_out


def project_fp8_workspace(m: int, n: int, k: int, dtype=torch.float32, device="cuda:0", stream=None):
    """Workspace of ngram_project_fp8 for C [m][n] of ``dtype`` over k
    columns, on ``stream`` (by default the current one), or None where the
    call needs none."""
    nbytes = lib().ngram_project_fp8_workspace_bytes(m, n, max(k, 1), F32 if dtype is torch.float32 else BF16)
    if nbytes < 0:
        raise NgramError(f"no 8-bit product has m={m}, n={n}, k={k}")
    return _new(nbytes, None, torch.uint8, device, stream) if nbytes else None


def ngram_project_fp8(a: Fp8, b: Fp8, out=None, dtype=torch.bfloat16, workspace=None, stream=None):
    """out [a.rows][b.rows] (fp32 or bf16) = a b^T over their common columns
    (of none, as in the weight gradient of an empty batch: zeros).
    A bf16 result of more than 32 rows keeps 13 bits below the largest product
    of each eight columns, an fp32 result everything (see ngram_project_fp8 in
    ngram.h)."""
    m, n = a.rows, b.rows
    if out is None:
        out = _new(m, n, dtype, a.codes.device, stream)
    po = _arg(out, _VALUES, m * n, "out")
    if a.cols == 0 and b.cols == 0 and n > 0 and n % 8 == 0:
        with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
            out.view(-1)[:m * n].zero_()
        return out
    if workspace is None:
        workspace = project_fp8_workspace(m, n, a.cols, out.dtype, out.device, stream)
    ws, ws_bytes = (None, 0) if workspace is None else _scratch(workspace)
    rc = lib().ngram_project_fp8(a.c, b.c, po, _value(out), ws, ws_bytes, _raw_stream(stream))
    if rc:
        _check(rc, "ngram_project_fp8")
    return out


def _step_c(step, lr, beta1, beta2, eps, weight_decay, grad_scale, seed):
    return _AdamWStep(lr, beta1, beta2, eps, weight_decay, grad_scale, step, seed & 0xFFFFFFFFFFFFFFFF)


def _adamw_tensor(p, g, m, v, m_scale, v_scale, rng_offset, name, g_numel=None, scale_bytes=None):
    n = p.numel()
    pp = _arg(p, _VALUES, n, f"{name}: p")
    pg = _arg(g, _VALUES, n if g_numel is None else g_numel, f"{name}: g")
    if m.dtype is torch.float32:
        if m_scale is not None or v_scale is not None:
            raise NgramError(f"{name}: fp32 moments have no scales")
        kinds, state, pms, pvs = _F32, STATE_F32, None, None
    else:
        kinds, state = _CODES, STATE_FP8
        need = -(-n // FP8_BLOCK) if scale_bytes is None else scale_bytes
        pms, pvs = _arg(m_scale, _BYTES, need, f"{name}: m_scale"), _arg(v_scale, _BYTES, need, f"{name}: v_scale")
    return _AdamWTensor(pp, pg, _arg(m, kinds, n, f"{name}: m"), _arg(v, kinds, n, f"{name}: v"), pms, pvs, n, rng_offset,
                        _value(p), _value(g), state, 0)


class AdamWTensors:
    """The tensors of ngram_adamw: equal-length lists of parameters (fp32 or
    bf16), gradients (fp32 or bf16) and moments, fp32 or 8-bit codes with
    ``m_scales`` and ``v_scales`` (uint8, one byte per 128 elements).

    The list names memory, and keeps that memory: a step reads the gradients
    and updates the parameters that were given here, whatever their names stand
    for by then.  Build it again when a gradient or another of them is a new
    tensor or has new memory (``p.data = ...``).  A program that lets its
    gradients go builds it each step; one that keeps and refills them (as it
    has to for a captured graph) does so once.  ``rng_offsets``: each tensor's
    place in the random sequence (by default one after the other, each at a
    multiple of 128)."""

    def __init__(self, params, grads, m, v, m_scales=None, v_scales=None, rng_offsets=None):
        count = len(params)
        none = [None] * count
        m_scales, v_scales = m_scales or none, v_scales or none
        if rng_offsets is None:
            rng_offsets, at = [], 0
            for p in params:
                rng_offsets.append(at)
                at += -(-p.numel() // FP8_BLOCK) * FP8_BLOCK
        lists = (params, grads, m, v, m_scales, v_scales, rng_offsets)
        if any(len(x) != count for x in lists):
            raise NgramError("the lists must have one entry for each parameter")
        self.tensors = [tuple(x) for x in zip(*lists[:6])]
        self.count = count
        self.c = (_AdamWTensor * max(count, 1))(*[_adamw_tensor(*x, name=f"tensor {i}") for i, x in enumerate(zip(*lists))])
        # a tensor may be given other memory (p.data = ...) while this list lives
        self.storages = [t.untyped_storage() for x in self.tensors for t in x if t is not None]


def ngram_adamw(tensors: AdamWTensors, lr, step, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, grad_scale=1.0,
                seed=0, stream=None):
    """One AdamW step on every tensor, in place; ``step`` counts from 1 (see
    ngram_adamw in ngram.h)."""
    rc = lib().ngram_adamw(tensors.c, tensors.count, _step_c(step, lr, beta1, beta2, eps, weight_decay, grad_scale, seed),
                           _raw_stream(stream))
    if rc:
        _check(rc, "ngram_adamw")


def ngram_adamw_rows(p, m, v, rows, g, n_rows=None, m_scale=None, v_scale=None, *, lr, step, beta1=0.9, beta2=0.999,
                     eps=1e-8, weight_decay=0.0, grad_scale=1.0, seed=0, stream=None):
    """One AdamW step on rows ``rows`` of the table p [R][d] from the sparse
    gradient (rows, g [max_rows][d], n_rows [1] int64 on the device) that
    ngram_grad_table and ngram_grad_e1 return (see ngram_adamw_rows in
    ngram.h).  Two tables, or a table and the tensors of ngram_adamw, round
    alike at equal places under one ``seed``: give each its own."""
    R, d = _matrix(p, "p")
    max_rows = 0 if rows is None else rows.numel()
    pr, pn = _arg(rows, _I32T, 0, "rows"), _opt(n_rows, (torch.int64,), 1, "n_rows")
    t = _adamw_tensor(p, g, m, v, m_scale, v_scale, 0, "table", g_numel=max_rows * d, scale_bytes=R * -(-d // FP8_BLOCK))
    rc = lib().ngram_adamw_rows(t, R, d, pr, max_rows, pn, _step_c(step, lr, beta1, beta2, eps, weight_decay, grad_scale, seed),
                                _raw_stream(stream))
    if rc:
        _check(rc, "ngram_adamw_rows")


INT4_GROUPS = (32, 64, 128)
INT4_MAX_ROWS = 1 << 24
INT4_MAX_COLS = 1 << 20
MAX_BEAMS = 32
DISTILL_MAX_K = 1024

_MARKS = (torch.bool, torch.uint8)


def _here(stream, *tensors):
    """Refuse tensors of another device than the current one, on whose queue the call goes."""
    d = torch._C._cuda_getDevice()
    for t in tensors:
        if t is not None and t.get_device() != d:
            raise NgramError(f"a tensor of {t.device} in a call on cuda:{d}: make its device the current one")
    if stream is not None and stream.device_index != d:
        raise NgramError(f"a stream of cuda:{stream.device_index} in a call on cuda:{d}")


def _one_device(*tensors):
    """Refuse tensors that are meant to be used together but lie on several devices."""
    if len({t.get_device() for t in tensors if t is not None}) > 1:
        raise NgramError("the tensors lie on several devices")


def _rows_arg(t, dtypes, name):
    """(pointer, rows, columns, distance of rows in elements) of a device matrix whose rows are contiguous."""
    n, v = _matrix(t, name)
    if t.dtype not in dtypes or not t.is_cuda:
        _dev(t, dtypes, name)
    sn, sv = t.stride()
    if sv != 1 and v > 1:
        raise NgramError(f"the rows of {name} must be contiguous")
    if sn < v:
        if n > 1:
            raise NgramError(f"the rows of {name} overlap")
        sn = v
    return t.data_ptr(), n, v, sn


class Int4:
    """A matrix in 4 bits: ``codes`` [rows][16 ceil(cols / 32)] bytes, ``scales`` (fp32 or bf16) and optionally ``zeros``
    (bytes) [rows][4 ceil(ceil(cols / group) / 4)]; see "4-bit matrices" in ngram.h.  It keeps its tensors."""

    __slots__ = ("codes", "scales", "zeros", "rows", "cols", "group", "c")

    def __init__(self, codes, scales, rows: int, cols: int, group: int = 128, zeros=None):
        ld, sld = _int4_shape(rows, cols, group)
        self.rows, self.cols, self.group = rows, cols, group
        self.codes, self.scales, self.zeros = codes, scales, zeros
        _one_device(codes, scales, zeros)
        self.c = _Int4(_arg(codes, (torch.uint8,), rows * ld, "codes"), _arg(scales, _VALUES, rows * sld, "scales"),
                       _opt(zeros, (torch.uint8,), rows * sld, "zeros"), rows, cols, group, _value(scales))

    @classmethod
    def empty(cls, rows: int, cols: int, group: int = 128, zeros: bool = True, scale_dtype=torch.bfloat16, device="cuda:0",
              stream=None) -> "Int4":
        if torch.device(device).type != "cuda":
            raise NgramError(f"a 4-bit matrix lies on a GPU, not on device {device}")
        if scale_dtype not in (torch.float32, torch.bfloat16):
            raise NgramError(f"scales are fp32 or bf16, not {scale_dtype}")
        return cls._empty(rows, cols, group, zeros, scale_dtype, device, stream)

    @classmethod
    def _empty(cls, rows, cols, group, zeros, scale_dtype, device, stream):
        ld, sld = _int4_shape(rows, cols, group)
        self = cls.__new__(cls)
        self.rows, self.cols, self.group = rows, cols, group
        self.codes, self.scales = _new(rows, ld, torch.uint8, device, stream), _new(rows, sld, scale_dtype, device, stream)
        self.zeros = _new(rows, sld, torch.uint8, device, stream) if zeros else None
        self.c = _Int4(self.codes.data_ptr(), self.scales.data_ptr(), self.zeros.data_ptr() if zeros else None, rows, cols, group,
                       _value(self.scales))
        return self


def _int4_shape(rows, cols, group):
    """(code bytes a row, scales a row), as ngram_int4_code_bytes and ngram_int4_scales count them."""
    if not (0 <= rows <= INT4_MAX_ROWS and 0 <= cols <= INT4_MAX_COLS) or cols % 8 or group not in INT4_GROUPS:
        raise NgramError(f"no 4-bit matrix has rows={rows}, cols={cols}, group={group}")
    return (cols + 31) // 32 * 16, ((cols + group - 1) // group + 3) // 4 * 4


def ngram_quant_int4(x, group: int = 128, zeros: bool = True, scale_dtype=torch.bfloat16, out: Optional[Int4] = None, stream=None) -> Int4:
    """x [n][d] (fp32 or bf16) in 4 bits (see ngram_quant_int4 in ngram.h); ``out``: the Int4 to fill, whose group, zeros
    and scales' type then count."""
    n, d = _matrix(x, "x")
    px = _arg(x, _VALUES, n * d, "x")
    if out is None:
        _here(stream, x)
        if scale_dtype not in (torch.float32, torch.bfloat16):
            raise NgramError(f"scales are fp32 or bf16, not {scale_dtype}")
        out = Int4._empty(n, d, group, zeros, scale_dtype, x.device, stream)
    else:
        _here(stream, x, out.codes)
    rc = lib().ngram_quant_int4(px, _value(x), n, d, out.c, _raw_stream(stream))
    if rc:
        _check(rc, "ngram_quant_int4")
    return out


def ngram_dequant_int4(q: Int4, out=None, dtype=torch.float32, stream=None):
    """The values of q, [q.rows][q.cols] fp32 or bf16 (see ngram_dequant_int4 in ngram.h)."""
    _here(stream, q.codes, out)
    if out is None:
        out = _new(q.rows, q.cols, dtype, q.codes.device, stream)
    rc = lib().ngram_dequant_int4(q.c, _arg(out, _VALUES, q.rows * q.cols, "out"), _value(out), _raw_stream(stream))
    if rc:
        _check(rc, "ngram_dequant_int4")
    return out


def ngram_project_int4(x, w: Int4, out=None, dtype=torch.bfloat16, stream=None):
    """out [n][w.rows] (fp32 or bf16) = x w^T for x [n][w.cols] (fp32 or bf16; see ngram_project_int4 in ngram.h)."""
    n, k = _matrix(x, "x")
    if k != w.cols:
        raise NgramError(f"x has {k} columns and w {w.cols}")
    px = _arg(x, _VALUES, n * k, "x")
    _here(stream, x, w.codes, out)
    if out is None:
        out = _new(n, w.rows, dtype, x.device, stream)
    rc = lib().ngram_project_int4(px, _value(x), n, w.c, _arg(out, _VALUES, n * w.rows, "out"), _value(out), _raw_stream(stream))
    if rc:
        _check(rc, "ngram_project_int4")
    return out


class BeamOut(NamedTuple):
    """ngram_beam_step's outputs, one entry (history: two) for each row; None for those not asked for."""
    scores: torch.Tensor
    tokens: Optional[torch.Tensor]
    parents: torch.Tensor
    history: Optional[torch.Tensor]
    finished: Optional[torch.Tensor]


def beam_step_workspace(batch: int, beams: int, V: int, dtype=torch.float32, device="cuda:0", stream=None):
    """Workspace of ngram_beam_step, on ``stream`` (by default the current one)."""
    nbytes = lib().ngram_beam_step_workspace_bytes(batch, beams, V, F32 if dtype is torch.float32 else BF16)
    if nbytes < 0:
        raise NgramError(f"no beam step has batch={batch}, beams={beams}, V={V}")
    return _new(nbytes, None, torch.uint8, device, stream)


def ngram_beam_step(logits, scores, beams: int, tokens=None, history=None, finished=None, end_token: int = -1,
                    out: Optional[BeamOut] = None, workspace=None, stream=None) -> BeamOut:
    """The next beams of every sequence from logits [batch * beams][V] (fp32 or bf16; rows at any distance) and the beams'
    scores (see ngram_beam_step in ngram.h).  ``tokens``, the tokens fed at this step, and ``history`` [rows][2], what
    ngram_forward took with them, give the next history; ``finished`` (bool or uint8) marks beams that have ended.
    ``out``: where to write, whose tensors may be the inputs of the same names; a None there is not written."""
    pl, rows, V, ld = _rows_arg(logits, _VALUES, "logits")
    if beams < 1 or rows % beams:
        raise NgramError(f"{rows} rows of logits are no whole sequences of {beams} beams")
    batch = rows // beams
    _here(stream, logits, scores, tokens, history, finished, workspace)
    if out is None:
        dev = logits.device
        out = BeamOut(_new(rows, None, torch.float32, dev, stream), _new(rows, None, torch.int32, dev, stream),
                      _new(rows, None, torch.int32, dev, stream), None if history is None else _new(rows, 2, torch.int32, dev, stream),
                      _new(rows, None, torch.bool, dev, stream) if end_token >= 0 else None)
    else:
        _here(stream, *out)
    if workspace is None:
        workspace = beam_step_workspace(batch, beams, V, logits.dtype, logits.device, stream)
    ws, ws_bytes = _scratch(workspace)
    rc = lib().ngram_beam_step(pl, _value(logits), batch, beams, V, ld, _arg(scores, _F32, rows, "scores"),
                               _opt(tokens, _I32T, rows, "tokens"), _opt(history, _I32T, 2 * rows, "history"),
                               _opt(finished, _MARKS, rows, "finished"), end_token, _arg(out.scores, _F32, rows, "out.scores"),
                               _opt(out.tokens, _I32T, rows, "out.tokens"), _arg(out.parents, _I32T, rows, "out.parents"),
                               _opt(out.history, _I32T, 2 * rows, "out.history"), _opt(out.finished, _MARKS, rows, "out.finished"),
                               ws, ws_bytes, _raw_stream(stream))
    if rc:
        _check(rc, "ngram_beam_step")
    return out


def _apart(states, rows):
    """Refuse (address, bytes of a row, distance of rows) of which two share bytes; rows that interleave do not."""
    begun = []
    for at, row, stride in sorted(s for s in states if s[1] > 0 and rows > 0):
        begun = [b for b in begun if b[0] + (rows - 1) * b[2] + b[1] > at]
        for first, size, step in begun:
            off = (at - first) % stride
            if step != stride or off < size or stride - off < row:
                raise NgramError("two states overlap")
        begun.append((at, row, stride))


class BeamStates:
    """The tensors that ngram_beam_reorder moves: each has the rows of all beams as its first dimension (at any distance),
    and contiguous rows; no two share memory.  The list names memory, and keeps that memory."""

    def __init__(self, tensors):
        self.tensors = list(tensors)
        rows = {t.shape[0] for t in self.tensors if t.dim() > 0}
        if any(t.dim() == 0 for t in self.tensors) or len(rows) > 1:
            raise NgramError("every state must have the same rows as its first dimension")
        self.rows = rows.pop() if rows else 0
        _one_device(*self.tensors)
        c = []
        for i, t in enumerate(self.tensors):
            if not t.is_cuda:
                raise NgramError(f"state {i} must be a device tensor")
            if self.rows > 0 and not t[0].is_contiguous():
                raise NgramError(f"state {i}: its rows must be contiguous")
            size = t.element_size()
            row = t.numel() // max(self.rows, 1) * size
            stride = t.stride(0) * size if self.rows > 1 else row
            if stride < row:
                raise NgramError(f"state {i}: its rows overlap")
            c.append(_BeamState(t.data_ptr(), row, stride))
        _apart([(s.data, s.row_bytes, s.stride) for s in c], self.rows)
        self.count = len(c)
        self.c = (_BeamState * max(self.count, 1))(*c)
        self.storages = [t.untyped_storage() for t in self.tensors]


def ngram_beam_reorder(states: BeamStates, parents, beams: int, stream=None):
    """Every state's row of a beam takes the row of the beam's parent, in place (see ngram_beam_reorder in ngram.h);
    ``parents`` as ngram_beam_step returns them."""
    rows = parents.numel()
    if beams < 1 or rows % beams or (states.count and rows != states.rows):
        raise NgramError(f"{rows} parents for {states.rows} rows of {beams} beams a sequence")
    _here(stream, parents, *states.tensors[:1])
    rc = lib().ngram_beam_reorder(states.c, states.count, _arg(parents, _I32T, rows, "parents"), rows // beams, beams, _raw_stream(stream))
    if rc:
        _check(rc, "ngram_beam_reorder")


class DistillOut(NamedTuple):
    """ngram_distill's outputs; None for those not asked for."""
    loss: Optional[torch.Tensor]
    stats: Optional[torch.Tensor]
    dlogits: Optional[torch.Tensor]


def distill_workspace(n: int, V: int, k: int, dtype=torch.float32, device="cuda:0", stream=None):
    """Workspace of ngram_distill, on ``stream`` (by default the current one)."""
    nbytes = lib().ngram_distill_workspace_bytes(n, V, k, F32 if dtype is torch.float32 else BF16)
    if nbytes < 0:
        raise NgramError(f"no distillation has n={n}, V={V}, k={k}")
    return _new(nbytes, None, torch.uint8, device, stream)


def _distill_args(logits, teacher, ids, temperature, teacher_lse):
    pz, n, V, ld = _rows_arg(logits, _VALUES, "logits")
    rows, k = _matrix(teacher, "teacher")
    if rows != n or ids is None or ids.shape != teacher.shape:
        raise NgramError("teacher and ids must have a row for each row of logits, and equal shapes")
    return _DistillArgs(pz, _arg(teacher, _VALUES, n * k, "teacher"), _arg(ids, _I32T, n * k, "ids"), _opt(teacher_lse, _F32, n, "teacher_lse"),
                        n, V, ld, k, _value(logits), _value(teacher), temperature)


def _dlogits(logits, n, V, dlogits_out, stream):
    """(tensor, pointer, distance of rows) of the gradient's buffer."""
    if dlogits_out is None:
        dlogits_out = _new(n, V, logits.dtype, logits.device, stream)
        return dlogits_out, dlogits_out.data_ptr(), V
    p, rows, cols, ld = _rows_arg(dlogits_out, (logits.dtype,), "dlogits_out")
    if rows != n or cols != V:
        raise NgramError(f"dlogits_out is {rows} x {cols}, logits {n} x {V}")
    return dlogits_out, p, ld


def ngram_distill(logits, teacher, ids, temperature: float = 1.0, teacher_lse=None, grad: bool = False, weight=None, scale: float = 1.0,
                  keep_stats: bool = False, loss_out=None, stats_out=None, dlogits_out=None, workspace=None, stream=None) -> DistillOut:
    """Loss [n] fp32 of the student's logits [n][V] against the teacher's top logits ``teacher`` [n][k] at tokens ``ids``
    [n][k] (see ngram_distill in ngram.h), and with ``grad`` or ``dlogits_out`` (which may be ``logits``) the gradient of the
    sum of weight * scale * loss in the same call.  ``keep_stats``: what ngram_distill_grad reads."""
    a = _distill_args(logits, teacher, ids, temperature, teacher_lse)
    n, V, dev = a.n, a.V, logits.device
    _here(stream, logits, teacher, ids, teacher_lse, weight, loss_out, stats_out, dlogits_out, workspace)
    if loss_out is None:
        loss_out = _new(n, None, torch.float32, dev, stream)
    if stats_out is None and keep_stats:
        stats_out = _new(n, 3, torch.float32, dev, stream)
    pd, dld = None, V
    if grad or dlogits_out is not None:
        dlogits_out, pd, dld = _dlogits(logits, n, V, dlogits_out, stream)
    if workspace is None:
        workspace = distill_workspace(n, V, a.k, logits.dtype, dev, stream)
    ws, ws_bytes = _scratch(workspace)
    rc = lib().ngram_distill(a, _arg(loss_out, _F32, n, "loss_out"), _opt(stats_out, _F32, 3 * n, "stats_out"),
                             _opt(weight, _F32, n, "weight"), scale, pd, dld, ws, ws_bytes, _raw_stream(stream))
    if rc:
        _check(rc, "ngram_distill")
    return DistillOut(loss_out, stats_out, dlogits_out)


def ngram_distill_grad(logits, teacher, ids, stats, temperature: float = 1.0, teacher_lse=None, weight=None, scale: float = 1.0,
                       dlogits_out=None, stream=None):
    """The gradient [n][V] of the sum of weight * scale * loss, from the forward's ``stats`` (see ngram_distill in ngram.h);
    ``dlogits_out`` may be ``logits``."""
    a = _distill_args(logits, teacher, ids, temperature, teacher_lse)
    _here(stream, logits, teacher, ids, stats, teacher_lse, weight, dlogits_out)
    dlogits_out, pd, dld = _dlogits(logits, a.n, a.V, dlogits_out, stream)
    rc = lib().ngram_distill_grad(a, _arg(stats, _F32, 3 * a.n, "stats"), _opt(weight, _F32, a.n, "weight"), scale, pd, dld,
                                  _raw_stream(stream))
    if rc:
        _check(rc, "ngram_distill_grad")
    return dlogits_out
