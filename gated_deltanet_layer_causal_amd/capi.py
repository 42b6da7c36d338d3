"""ctypes binding of libgdn.so: the C ABI in include/libgdn.h, one Python
function per exported entry point, same names.

Argument marshalling only: tensors are torch CUDA (HIP) tensors, passed as
raw device pointers with their row strides; the stream is torch's current
stream unless one is given.  All arithmetic happens in the HIP kernels.
There is no fallback: if the library is missing, was built from other
sources than those in the tree, or a call fails, an error is raised.

The C side takes most tensors without strides and cannot see their sizes, so
every wrapper checks dtype, device, layout and element count against the
shape before the call: a caller's mistake becomes a Python exception rather
than an out-of-bounds device access.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from ctypes import POINTER, byref, c_float, c_int, c_int32, c_int64, c_size_t, c_void_p

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdn.so")

GDN_BF16, GDN_FP32, GDN_FP16 = 0, 1, 2
GDN_ACT_SILU, GDN_ACT_SIGMOID = 0, 1
EXPORTS = (
    "gdn_status_string", "gdn_conv_fwd", "gdn_conv_bwd", "gdn_conv_bwd_workspace",
    "gdn_conv_bwd_noalloc", "gdn_conv_fwd_state", "gdn_conv_bwd_state", "gdn_gate_fwd",
    "gdn_gate_bwd", "gdn_gate_bwd_workspace", "gdn_chunk_fwd", "gdn_chunk_fwd_workspace",
    "gdn_chunk_bwd", "gdn_chunk_bwd_workspace", "gdn_gated_norm_fwd", "gdn_gated_norm_bwd",
    "gdn_gated_norm_bwd_workspace", "gdn_chunk_prepare", "gdn_chunk_prepare_bwd",
    "gdn_chunk_fwd_states", "gdn_chunk_fwd_states_save",
    "gdn_chunk_bwd_states", "gdn_chunk_bwd_reverse", "gdn_chunk_bwd_grads",
    "gdn_check_cu_seqlens", "gdn_recurrent_fwd", "gdn_step_fwd", "gdn_check_slots",
    "gdn_cache_copy", "gdn_cache_fork", "gdn_cache_retain", "gdn_cache_release",
    "gdn_cache_compact", "gdn_cache_workspace",
)


class Shape(ctypes.Structure):
    _fields_ = [("n_seq", c_int32), ("total_tokens", c_int64), ("hk", c_int32), ("hv", c_int32),
                ("dk", c_int32), ("dv", c_int32), ("conv_k", c_int32), ("chunk", c_int32),
                ("dtype", c_int), ("seg_chunks", c_int32)]


class Cache(ctypes.Structure):
    """gdn_cache: the slots of one layer's states.  Made by make_cache, which
    checks the tensors and keeps them (`S`, `conv`)."""
    _fields_ = [("S_ptr", c_void_p), ("S_stride", c_int64), ("conv_ptr", c_void_p),
                ("conv_stride", c_int64), ("n_slots", c_int32)]


class GDNError(RuntimeError):
    def __init__(self, name, status, msg):
        super().__init__(f"{name} failed: status {status} ({msg})")
        self.status = status


_lib = None


def _check_built(path: str):
    from . import build as _b
    hint = "build it first: python -c 'import __graft_entry__ as g; g.build()'"
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing; {hint}")
    dig = path + ".sources"
    have = open(dig).read().strip() if os.path.exists(dig) else None
    if have != _b.source_digest():
        raise RuntimeError(f"{path} was not built from the HIP sources in this tree; {hint}")


def load(path: str = LIB_PATH):
    """Load libgdn.so; refuses a missing library or one built from other
    sources (the digest written by build.py must match csrc/ and include/)."""
    global _lib
    if _lib is not None:
        return _lib
    _check_built(path)
    lib = ctypes.CDLL(path)
    SP = POINTER(Shape)
    V, I64, F = c_void_p, c_int64, c_float
    lib.gdn_status_string.argtypes = [c_int]
    lib.gdn_status_string.restype = ctypes.c_char_p
    lib.gdn_conv_fwd.argtypes = [SP, V, I64, V, V, c_int, F, V, I64, V]
    lib.gdn_conv_bwd.argtypes = [SP, V, I64, V, V, c_int, F, V, I64, V, I64, V, V, c_size_t, V]
    lib.gdn_conv_bwd_noalloc.argtypes = [SP, V, I64, V, V, c_int, F, V, I64, V, I64, V, V]
    lib.gdn_conv_fwd_state.argtypes = [SP, V, I64, V, V, c_int, F, V, V, I64, V, V]
    lib.gdn_conv_bwd_state.argtypes = [SP, V, I64, V, V, c_int, F, V, V, I64, V, V, I64, V, V, V,
                                       c_size_t, V]
    lib.gdn_gate_fwd.argtypes = [SP, V, V, V, V, V, V, V]
    lib.gdn_gate_bwd.argtypes = [SP, V, V, V, V, V, V, V, V, V, V, V, c_size_t, V]
    lib.gdn_chunk_fwd.argtypes = [SP, V, V, V, I64, I64, I64, V, V, F, V, V, V, V, V, c_size_t, V]
    lib.gdn_chunk_bwd.argtypes = [SP, V, V, V, I64, I64, I64, V, V, F, V, V, V, V, V, V, V, I64,
                                  I64, I64, V, V, V, V, c_size_t, V]
    lib.gdn_chunk_prepare.argtypes = [SP, V, V, I64, I64, V, V, F, V, V, c_size_t, V]
    lib.gdn_chunk_prepare_bwd.argtypes = [SP, V, V, I64, I64, V, V, F, V, V, c_size_t, V]
    lib.gdn_chunk_fwd_states.argtypes = [SP, V, V, V, I64, I64, I64, F, V, V, V, V, V, c_size_t, V]
    lib.gdn_chunk_fwd_states_save.argtypes = lib.gdn_chunk_fwd_states.argtypes
    lib.gdn_chunk_bwd_states.argtypes = [SP, V, V, V, I64, I64, I64, F, V, V, V, c_size_t, V]
    lib.gdn_chunk_bwd_reverse.argtypes = [SP, V, V, I64, I64, F, V, V, V, V, I64, V, V, c_size_t, V]
    lib.gdn_chunk_bwd_grads.argtypes = [SP, V, V, I64, I64, V, F, V, V, V, I64, V, V, I64, I64, V,
                                        V, V, c_size_t, V]
    lib.gdn_gated_norm_fwd.argtypes = [I64, c_int32, c_int, V, V, V, F, c_int, V, V]
    lib.gdn_check_cu_seqlens.argtypes = [SP, V, V, V]
    lib.gdn_gated_norm_bwd.argtypes = [I64, c_int32, c_int, V, V, V, F, c_int, V, V, V, V, V,
                                       c_size_t, V]
    CP, I32 = POINTER(Cache), c_int32
    lib.gdn_recurrent_fwd.argtypes = [SP, V, V, V, I64, I64, I64, V, V, F, CP, V, V, V, V, V, V]
    lib.gdn_step_fwd.argtypes = [SP, V, I64, V, V, I64, V, I64, V, V, V, I64, V, F, F, F, c_int, CP,
                                 V, V, V, V, V, V]
    lib.gdn_check_slots.argtypes = [SP, I32, V, V, V, V, V, V]
    lib.gdn_cache_copy.argtypes = [V, I64, I32, V, V, I64, I32, V, I64, I32, V]
    lib.gdn_cache_fork.argtypes = [V, I64, I32, V, V, I32, V, V, c_size_t, V]
    lib.gdn_cache_retain.argtypes = [V, I32, V, I32, V]
    lib.gdn_cache_release.argtypes = [V, I32, V, I32, V]
    lib.gdn_cache_compact.argtypes = [V, I64, I32, V, V, V, I32, V, c_size_t, V]
    lib.gdn_cache_workspace.argtypes = [I32]
    lib.gdn_cache_workspace.restype = c_size_t
    for name in ("gdn_conv_bwd_workspace", "gdn_gate_bwd_workspace", "gdn_chunk_fwd_workspace",
                 "gdn_chunk_bwd_workspace"):
        getattr(lib, name).argtypes = [SP]
        getattr(lib, name).restype = c_size_t
    lib.gdn_gated_norm_bwd_workspace.argtypes = [I64, c_int32]
    lib.gdn_gated_norm_bwd_workspace.restype = c_size_t
    for name in ("gdn_conv_fwd", "gdn_conv_bwd", "gdn_conv_bwd_noalloc", "gdn_conv_fwd_state",
                 "gdn_conv_bwd_state", "gdn_gate_fwd", "gdn_gate_bwd", "gdn_chunk_fwd",
                 "gdn_chunk_bwd", "gdn_gated_norm_fwd", "gdn_gated_norm_bwd", "gdn_chunk_prepare",
                 "gdn_chunk_prepare_bwd", "gdn_chunk_fwd_states", "gdn_chunk_fwd_states_save",
                 "gdn_chunk_bwd_states", "gdn_chunk_bwd_reverse",
                 "gdn_chunk_bwd_grads", "gdn_check_cu_seqlens", "gdn_recurrent_fwd", "gdn_step_fwd",
                 "gdn_check_slots", "gdn_cache_copy", "gdn_cache_fork", "gdn_cache_retain",
                 "gdn_cache_release", "gdn_cache_compact"):
        getattr(lib, name).restype = c_int
    _lib = lib
    return lib


def _p(t):
    """The device pointer of a tensor (None for None); host tensors are
    refused here, after the wrappers' dtype and size checks."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libgdn takes device tensors only; got a host tensor")
    return c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return c_void_p(s.cuda_stream)


def _ok(name, st):
    if st != 0:
        raise GDNError(name, st, load().gdn_status_string(st).decode())


_GDN_DT = {torch.bfloat16: GDN_BF16, torch.float32: GDN_FP32, torch.float16: GDN_FP16}


def _dt(t: torch.Tensor) -> int:
    if t.dtype not in _GDN_DT:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return _GDN_DT[t.dtype]


def make_shape(n_seq, total_tokens, hk, hv, d, dtype, seg_chunks=0) -> Shape:
    """seg_chunks: segment length of the segment-parallel state scan (0: the
    library decides, > 0: forced, < 0: one sequential pass per sequence)."""
    dt = dtype if isinstance(dtype, int) else _GDN_DT[dtype]
    return Shape(n_seq, total_tokens, hk, hv, d, d, 4, 64, dt, seg_chunks)


def _ld(t):
    return t.stride(0) if t.dim() > 0 else 0


# ---------------------------------------------------------------- workspace queries
def gdn_conv_bwd_workspace(shape):
    return int(load().gdn_conv_bwd_workspace(byref(shape)))


def gdn_gate_bwd_workspace(shape):
    return int(load().gdn_gate_bwd_workspace(byref(shape)))


def gdn_chunk_fwd_workspace(shape):
    return int(load().gdn_chunk_fwd_workspace(byref(shape)))


def gdn_chunk_bwd_workspace(shape):
    return int(load().gdn_chunk_bwd_workspace(byref(shape)))


def gdn_gated_norm_bwd_workspace(rows, dv):
    return int(load().gdn_gated_norm_bwd_workspace(rows, dv))


# ---------------------------------------------------------------- argument checks
_TDT = {GDN_BF16: torch.bfloat16, GDN_FP32: torch.float32, GDN_FP16: torch.float16}


def _tdt(shape) -> torch.dtype:
    return _TDT[shape.dtype]


def _need(name, t, dtype, numel=None, optional=False):
    """A contiguous device tensor of `dtype` with `numel` elements (or None
    when optional)."""
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, the shape needs {numel}")


def _rows(name, t, dtype, T, cols):
    """A [T, cols] device matrix of `dtype` with contiguous rows (any row
    stride; the C side checks its alignment)."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2 or tuple(t.shape) != (T, cols) or (T > 0 and cols > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be a [{T}, {cols}] matrix with contiguous rows, got "
                         f"shape {tuple(t.shape)} strides {t.stride()}")


def _ws(ws):
    if ws is None:
        return
    if ws.dtype != torch.uint8 or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")


def _cu_ok(shape, cu):
    _need("cu_seqlens", cu, torch.int32, shape.n_seq + 1)


def _state(name, shape, t, optional=True):
    _need(name, t, torch.float32, shape.n_seq * shape.hv * shape.dk * shape.dv, optional=optional)


def _chunk_qk(shape, q, k):
    _rows("q", q, _tdt(shape), shape.total_tokens, shape.hk * shape.dk)
    _rows("k", k, _tdt(shape), shape.total_tokens, shape.hk * shape.dk)


def _per_token(name, shape, t, dtype=torch.float32):
    _need(name, t, dtype, shape.total_tokens * shape.hv)


def _heads(name, shape, t):
    _need(name, t, _tdt(shape), shape.total_tokens * shape.hv * shape.dv)


def _conv_ok(shape, x, w, cu):
    C = 2 * shape.hk * shape.dk + shape.hv * shape.dv
    _rows("x", x, _tdt(shape), shape.total_tokens, C)
    _need("w", w, torch.float32, C * 4)
    _cu_ok(shape, cu)
    return C


# ---------------------------------------------------------------- entry points
def gdn_conv_fwd(shape, x, w, cu_seqlens, y, l2norm_qk=True, l2_eps=1e-6, stream=None):
    C = _conv_ok(shape, x, w, cu_seqlens)
    _rows("y", y, _tdt(shape), shape.total_tokens, C)
    _ok("gdn_conv_fwd", load().gdn_conv_fwd(byref(shape), _p(x), _ld(x), _p(w), _p(cu_seqlens),
                                            int(l2norm_qk), l2_eps, _p(y), _ld(y), _stream(stream)))


def gdn_conv_bwd(shape, x, w, cu_seqlens, dy, dx, dw, ws, l2norm_qk=True, l2_eps=1e-6,
                 stream=None):
    C = _conv_ok(shape, x, w, cu_seqlens)
    _rows("dy", dy, _tdt(shape), shape.total_tokens, C)
    _rows("dx", dx, _tdt(shape), shape.total_tokens, C)
    _need("dw", dw, torch.float32, C * 4)
    _ws(ws)
    _ok("gdn_conv_bwd", load().gdn_conv_bwd(byref(shape), _p(x), _ld(x), _p(w), _p(cu_seqlens),
                                            int(l2norm_qk), l2_eps, _p(dy), _ld(dy), _p(dx),
                                            _ld(dx), _p(dw), _p(ws), ws.numel() if ws is not None else 0,
                                            _stream(stream)))


def _conv_state(name, shape, t):
    _need(name, t, _tdt(shape), shape.n_seq * 3 * (2 * shape.hk * shape.dk + shape.hv * shape.dv),
          optional=True)


def gdn_conv_fwd_state(shape, x, w, cu_seqlens, y, conv_state_in=None, conv_state_out=None,
                       l2norm_qk=True, l2_eps=1e-6, stream=None):
    C = _conv_ok(shape, x, w, cu_seqlens)
    _rows("y", y, _tdt(shape), shape.total_tokens, C)
    _conv_state("conv_state_in", shape, conv_state_in)
    _conv_state("conv_state_out", shape, conv_state_out)
    _ok("gdn_conv_fwd_state", load().gdn_conv_fwd_state(
        byref(shape), _p(x), _ld(x), _p(w), _p(cu_seqlens), int(l2norm_qk), l2_eps,
        _p(conv_state_in), _p(y), _ld(y), _p(conv_state_out), _stream(stream)))


def gdn_conv_bwd_state(shape, x, w, cu_seqlens, dy, dx, dw, ws, conv_state_in=None,
                       d_conv_state_out=None, d_conv_state_in=None, l2norm_qk=True, l2_eps=1e-6,
                       stream=None):
    C = _conv_ok(shape, x, w, cu_seqlens)
    _rows("dy", dy, _tdt(shape), shape.total_tokens, C)
    _rows("dx", dx, _tdt(shape), shape.total_tokens, C)
    _need("dw", dw, torch.float32, C * 4)
    for nm, t in (("conv_state_in", conv_state_in), ("d_conv_state_out", d_conv_state_out),
                  ("d_conv_state_in", d_conv_state_in)):
        _conv_state(nm, shape, t)
    _ws(ws)
    _ok("gdn_conv_bwd_state", load().gdn_conv_bwd_state(
        byref(shape), _p(x), _ld(x), _p(w), _p(cu_seqlens), int(l2norm_qk), l2_eps,
        _p(conv_state_in), _p(dy), _ld(dy), _p(d_conv_state_out), _p(dx), _ld(dx), _p(dw),
        _p(d_conv_state_in), _p(ws), ws.numel() if ws is not None else 0, _stream(stream)))


CONV_BWD_NOALLOC_MAX_BYTES = 32 << 20   # GDN_CONV_BWD_NOALLOC_MAX_BYTES in libgdn.h


def gdn_conv_bwd_noalloc(shape, x, w, cu_seqlens, dy, dx, dw, l2norm_qk=True, l2_eps=1e-6,
                         stream=None):
    """gdn_conv_bwd with the library's own scratch (no workspace, no
    allocation); see libgdn.h for its size limit and sharing rules."""
    C = _conv_ok(shape, x, w, cu_seqlens)
    _rows("dy", dy, _tdt(shape), shape.total_tokens, C)
    _rows("dx", dx, _tdt(shape), shape.total_tokens, C)
    _need("dw", dw, torch.float32, C * 4)
    _ok("gdn_conv_bwd_noalloc", load().gdn_conv_bwd_noalloc(
        byref(shape), _p(x), _ld(x), _p(w), _p(cu_seqlens), int(l2norm_qk), l2_eps, _p(dy),
        _ld(dy), _p(dx), _ld(dx), _p(dw), _stream(stream)))


def _gate_ok(shape, a, b, A_log, dt_bias):
    _per_token("a", shape, a, _tdt(shape))
    _per_token("b", shape, b, _tdt(shape))
    _need("A_log", A_log, torch.float32, shape.hv)
    _need("dt_bias", dt_bias, torch.float32, shape.hv)


CU_BAD_START, CU_BAD_END, CU_DECREASING = 1, 2, 4


def gdn_check_cu_seqlens(shape, cu_seqlens, violations, stream=None):
    """Writes to violations (an int32 device tensor of one element) the bit
    mask of the cu_seqlens contract's violations (CU_BAD_START, CU_BAD_END,
    CU_DECREASING; 0 when valid), asynchronously."""
    _cu_ok(shape, cu_seqlens)
    _need("violations", violations, torch.int32, 1)
    _ok("gdn_check_cu_seqlens", load().gdn_check_cu_seqlens(byref(shape), _p(cu_seqlens),
                                                            _p(violations), _stream(stream)))


def gdn_gate_fwd(shape, a, b, A_log, dt_bias, g, beta, stream=None):
    _gate_ok(shape, a, b, A_log, dt_bias)
    _per_token("g", shape, g)
    _per_token("beta", shape, beta)
    _ok("gdn_gate_fwd", load().gdn_gate_fwd(byref(shape), _p(a), _p(b), _p(A_log), _p(dt_bias),
                                            _p(g), _p(beta), _stream(stream)))


def gdn_gate_bwd(shape, a, b, A_log, dt_bias, dg, dbeta, da, db, dA_log, ddt_bias, ws,
                 stream=None):
    _gate_ok(shape, a, b, A_log, dt_bias)
    for nm, t in (("dg", dg), ("dbeta", dbeta)):
        _per_token(nm, shape, t)
    for nm, t in (("da", da), ("db", db)):
        _per_token(nm, shape, t, _tdt(shape))
    _need("dA_log", dA_log, torch.float32, shape.hv)
    _need("ddt_bias", ddt_bias, torch.float32, shape.hv)
    _ws(ws)
    _ok("gdn_gate_bwd", load().gdn_gate_bwd(byref(shape), _p(a), _p(b), _p(A_log), _p(dt_bias),
                                            _p(dg), _p(dbeta), _p(da), _p(db), _p(dA_log),
                                            _p(ddt_bias), _p(ws), ws.numel() if ws is not None else 0,
                                            _stream(stream)))


def _chunk_fwd_ok(shape, q, k, v, g, beta, S0, S_final, cu, o, ws):
    _chunk_qk(shape, q, k)
    _rows("v", v, _tdt(shape), shape.total_tokens, shape.hv * shape.dv)
    if g is not None or beta is not None:
        _per_token("g", shape, g)
        _per_token("beta", shape, beta)
    _state("S0", shape, S0)
    _state("S_final", shape, S_final)
    _cu_ok(shape, cu)
    if o is not None:
        _heads("o", shape, o)
    _ws(ws)


def gdn_chunk_fwd(shape, q, k, v, g, beta, scale, S0, S_final, cu_seqlens, o, ws, stream=None):
    _chunk_fwd_ok(shape, q, k, v, g, beta, S0, S_final, cu_seqlens, o, ws)
    _per_token("g", shape, g)
    _per_token("beta", shape, beta)
    _heads("o", shape, o)
    _ok("gdn_chunk_fwd", load().gdn_chunk_fwd(byref(shape), _p(q), _p(k), _p(v), _ld(q), _ld(k),
                                              _ld(v), _p(g), _p(beta), scale, _p(S0), _p(S_final),
                                              _p(cu_seqlens), _p(o), _p(ws), ws.numel(),
                                              _stream(stream)))


def _chunk_grads_ok(shape, dq, dk, dg, dbeta):
    _rows("dq", dq, _tdt(shape), shape.total_tokens, shape.hk * shape.dk)
    _rows("dk", dk, _tdt(shape), shape.total_tokens, shape.hk * shape.dk)
    _per_token("dg", shape, dg)
    _per_token("dbeta", shape, dbeta)


def gdn_chunk_bwd(shape, q, k, v, g, beta, scale, S0, cu_seqlens, dout, dS_final, dq, dk, dv, dg,
                  dbeta, dS0, ws, stream=None):
    _chunk_fwd_ok(shape, q, k, v, g, beta, S0, None, cu_seqlens, None, ws)
    _per_token("g", shape, g)
    _per_token("beta", shape, beta)
    _heads("dout", shape, dout)
    _state("dS_final", shape, dS_final)
    _state("dS0", shape, dS0)
    _chunk_grads_ok(shape, dq, dk, dg, dbeta)
    _rows("dv", dv, _tdt(shape), shape.total_tokens, shape.hv * shape.dv)
    _ok("gdn_chunk_bwd", load().gdn_chunk_bwd(byref(shape), _p(q), _p(k), _p(v), _ld(q), _ld(k),
                                              _ld(v), _p(g), _p(beta), scale, _p(S0),
                                              _p(cu_seqlens), _p(dout), _p(dS_final), _p(dq),
                                              _p(dk), _p(dv), _ld(dq), _ld(dk), _ld(dv), _p(dg),
                                              _p(dbeta), _p(dS0), _p(ws), ws.numel(),
                                              _stream(stream)))


def _prep_ok(shape, q, k, g, beta, cu, ws):
    _chunk_qk(shape, q, k)
    _per_token("g", shape, g)
    _per_token("beta", shape, beta)
    _cu_ok(shape, cu)
    _ws(ws)


def gdn_chunk_prepare(shape, q, k, g, beta, scale, cu_seqlens, ws, stream=None):
    _prep_ok(shape, q, k, g, beta, cu_seqlens, ws)
    _ok("gdn_chunk_prepare", load().gdn_chunk_prepare(byref(shape), _p(q), _p(k), _ld(q), _ld(k),
                                                      _p(g), _p(beta), scale, _p(cu_seqlens),
                                                      _p(ws), ws.numel(), _stream(stream)))


def gdn_chunk_prepare_bwd(shape, q, k, g, beta, scale, cu_seqlens, ws, stream=None):
    _prep_ok(shape, q, k, g, beta, cu_seqlens, ws)
    _ok("gdn_chunk_prepare_bwd", load().gdn_chunk_prepare_bwd(
        byref(shape), _p(q), _p(k), _ld(q), _ld(k), _p(g), _p(beta), scale, _p(cu_seqlens), _p(ws),
        ws.numel(), _stream(stream)))


def gdn_chunk_fwd_states(shape, q, k, v, scale, S0, S_final, cu_seqlens, o, ws, stream=None):
    _chunk_fwd_ok(shape, q, k, v, None, None, S0, S_final, cu_seqlens, o, ws)
    _heads("o", shape, o)
    _ok("gdn_chunk_fwd_states", load().gdn_chunk_fwd_states(
        byref(shape), _p(q), _p(k), _p(v), _ld(q), _ld(k), _ld(v), scale, _p(S0), _p(S_final),
        _p(cu_seqlens), _p(o), _p(ws), ws.numel(), _stream(stream)))


def gdn_chunk_fwd_states_save(shape, q, k, v, scale, S0, S_final, cu_seqlens, o, ws, stream=None):
    _chunk_fwd_ok(shape, q, k, v, None, None, S0, S_final, cu_seqlens, o, ws)
    _heads("o", shape, o)
    _ok("gdn_chunk_fwd_states_save", load().gdn_chunk_fwd_states_save(
        byref(shape), _p(q), _p(k), _p(v), _ld(q), _ld(k), _ld(v), scale, _p(S0), _p(S_final),
        _p(cu_seqlens), _p(o), _p(ws), ws.numel(), _stream(stream)))


def gdn_chunk_bwd_states(shape, q, k, v, scale, S0, cu_seqlens, ws, stream=None):
    _chunk_fwd_ok(shape, q, k, v, None, None, S0, None, cu_seqlens, None, ws)
    _ok("gdn_chunk_bwd_states", load().gdn_chunk_bwd_states(
        byref(shape), _p(q), _p(k), _p(v), _ld(q), _ld(k), _ld(v), scale, _p(S0), _p(cu_seqlens),
        _p(ws), ws.numel(), _stream(stream)))


def gdn_chunk_bwd_reverse(shape, q, k, scale, cu_seqlens, dout, dS_final, dv, dS0, ws, stream=None):
    _chunk_qk(shape, q, k)
    _cu_ok(shape, cu_seqlens)
    _heads("dout", shape, dout)
    _state("dS_final", shape, dS_final)
    _state("dS0", shape, dS0)
    _rows("dv", dv, _tdt(shape), shape.total_tokens, shape.hv * shape.dv)
    _ws(ws)
    _ok("gdn_chunk_bwd_reverse", load().gdn_chunk_bwd_reverse(
        byref(shape), _p(q), _p(k), _ld(q), _ld(k), scale, _p(cu_seqlens), _p(dout), _p(dS_final),
        _p(dv), _ld(dv), _p(dS0), _p(ws), ws.numel(), _stream(stream)))


def gdn_chunk_bwd_grads(shape, q, k, beta, scale, cu_seqlens, dout, dv, dq, dk, dg, dbeta, ws,
                        stream=None):
    _chunk_qk(shape, q, k)
    _per_token("beta", shape, beta)
    _cu_ok(shape, cu_seqlens)
    _heads("dout", shape, dout)
    _rows("dv", dv, _tdt(shape), shape.total_tokens, shape.hv * shape.dv)
    _chunk_grads_ok(shape, dq, dk, dg, dbeta)
    _ws(ws)
    _ok("gdn_chunk_bwd_grads", load().gdn_chunk_bwd_grads(
        byref(shape), _p(q), _p(k), _ld(q), _ld(k), _p(beta), scale, _p(cu_seqlens), _p(dout),
        _p(dv), _ld(dv), _p(dq), _p(dk), _ld(dq), _ld(dk), _p(dg), _p(dbeta), _p(ws), ws.numel(),
        _stream(stream)))


def _norm_ok(o, z, w, *others):
    dv = o.shape[-1]
    rows = o.numel() // dv if dv else 0
    dt = o.dtype
    _need("o", o, dt, rows * dv)
    _need("z", z, dt, rows * dv)
    for nm, t in others:
        _need(nm, t, dt, rows * dv)
    _need("w", w, torch.float32, dv)
    return rows, dv


def gdn_gated_norm_fwd(o, z, w, y, eps=1e-6, act=GDN_ACT_SILU, stream=None):
    rows, dv = _norm_ok(o, z, w, ("y", y))
    _ok("gdn_gated_norm_fwd", load().gdn_gated_norm_fwd(rows, dv, _dt(o), _p(o), _p(z), _p(w), eps,
                                                        act, _p(y), _stream(stream)))


def gdn_gated_norm_bwd(o, z, w, dy, dout, dz, dw, ws, eps=1e-6, act=GDN_ACT_SILU, stream=None):
    rows, dv = _norm_ok(o, z, w, ("dy", dy), ("dout", dout), ("dz", dz))
    _need("dw", dw, torch.float32, dv)
    _ws(ws)
    _ok("gdn_gated_norm_bwd", load().gdn_gated_norm_bwd(rows, dv, _dt(o), _p(o), _p(z), _p(w), eps,
                                                        act, _p(dy), _p(dout), _p(dz), _p(dw),
                                                        _p(ws), ws.numel(), _stream(stream)))


# ---------------------------------------------------------------- serving: cached states
def make_cache(S, conv=None) -> Cache:
    """The C ABI's gdn_cache from the slots' views: S fp32 [n_slots, hv, dv,
    dk] and (for the step) conv [n_slots, 3, C] in the storage type, each slot
    dense, any stride between slots."""
    if S.dtype != torch.float32 or S.dim() != 4 or S.shape[2] != S.shape[3] or S.shape[0] < 1:
        raise ValueError(f"S must be float32 [n_slots, hv, d, d], got {S.dtype} {tuple(S.shape)}")
    n, hv, d = S.shape[:3]
    if S.stride()[1:] != (d * d, d, 1):
        raise ValueError(f"each slot of S must be contiguous, got strides {S.stride()}")
    c = Cache(S.data_ptr(), S.stride(0) if n > 1 else hv * d * d, None, 0, n)
    c.conv_rows = None
    if conv is not None:
        if conv.dtype not in _GDN_DT or conv.dim() != 3 or tuple(conv.shape[:2]) != (n, 3):
            raise ValueError(f"conv must be [{n}, 3, C] in a storage type, got {conv.dtype} "
                             f"{tuple(conv.shape)}")
        C = conv.shape[2]
        if conv.stride()[1:] != (C, 1) or conv.device != S.device:
            raise ValueError("each slot of conv must be contiguous and on S's device")
        c.conv_ptr = conv.data_ptr()
        c.conv_stride = conv.stride(0) if n > 1 else 3 * C
        c.conv_rows = (conv.dtype, C)
    c.S, c.conv, c.device, c.index, c.heads = S, conv, S.device, S.get_device(), (hv, d)
    return c


# Serving calls are as short as a few microseconds, so their wrappers ask first
# whether every tensor is as it should be, as cheaply as Python can (one
# expression over dtype, shape, layout and device index), and go through the
# checks that say what is wrong only if one is not.
def _is_flat(t, dtype, numel, index):
    return (t.dtype is dtype and t.numel() == numel and t.get_device() == index >= 0 and
            t.is_contiguous())


_get_device = getattr(torch._C, "_cuda_getDevice", None)
_get_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(dev, index, stream):
    """The hipStream_t of `stream`, or of device `index`'s current one."""
    if index < 0:
        raise ValueError("libgdn takes device tensors only; got a host tensor")
    if stream is None:
        return _get_stream(index)
    if stream.device != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
    return stream.cuda_stream


def _run(name, index, args):
    """Runs a serving entry point on device `index`, which need not be the
    current one."""
    fn = getattr(_lib or load(), name)
    if index == _get_device():
        st = fn(*args)
    else:
        with torch.cuda.device(index):
            st = fn(*args)
    if st != 0:
        _ok(name, st)


def _on(dev, *named):
    for nm, t in named:
        if t is not None and t.device != dev:
            raise ValueError(f"{nm} is on {t.device}, the cache on {dev}")


def same_device(dev, **named):
    """ValueError naming the first tensor that is not on `dev`."""
    _on(dev, *named.items())


def current_device(dev):
    """A context with `dev` as the current device, for the entry points that
    run on the current device's stream (nothing to do where it is, nor for the
    host, whose tensors they refuse)."""
    if dev.type != "cuda" or dev.index == _get_device():
        return contextlib.nullcontext()
    return torch.cuda.device(dev)


def _slot_tables(shape, dev, cu, slot_in, slot_out, slot_tok):
    _cu_ok(shape, cu)
    _need("slot_in", slot_in, torch.int32, shape.n_seq, optional=True)
    _need("slot_out", slot_out, torch.int32, shape.n_seq, optional=True)
    _need("slot_tok", slot_tok, torch.int32, shape.total_tokens, optional=True)
    _on(dev, ("cu_seqlens", cu), ("slot_in", slot_in), ("slot_out", slot_out),
        ("slot_tok", slot_tok))


def _cache_ok(shape, cache):
    if cache.heads != (shape.hv, shape.dv):
        raise ValueError(f"the cache's states are of {cache.heads[0]} heads of {cache.heads[1]}, the "
                         f"shape's of {shape.hv} of {shape.dv}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _row_ld(t):
    """The row stride of a matrix; of fewer than two rows any serves (torch
    leaves a single row's stride open), so their width."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def gdn_recurrent_fwd(shape, q, k, v, g, beta, scale, cache, slot_in, slot_out, slot_tok,
                      cu_seqlens, o, stream=None):
    """cache: make_cache(S).  slot_in, slot_out [n_seq] and slot_tok [T]:
    int32 device tables, each may be None; see libgdn.h."""
    i, dt, T, N, hv, d = (cache.index, _TDT[shape.dtype], shape.total_tokens, shape.n_seq, shape.hv,
                          shape.dv)
    f32, i32, n = torch.float32, torch.int32, T * hv
    try:
        qs, ks, vs = q.stride(), k.stride(), v.stride()
        good = (T > 0 and i >= 0 and cache.heads == (hv, d) and
                q.dtype is dt and q.shape == (T, shape.hk * d) and qs[1] == 1 and q.get_device() == i and
                k.dtype is dt and k.shape == q.shape and ks[1] == 1 and k.get_device() == i and
                v.dtype is dt and v.shape == (T, hv * d) and vs[1] == 1 and v.get_device() == i and
                g.dtype is f32 and g.numel() == n and g.is_contiguous() and g.get_device() == i and
                beta.dtype is f32 and beta.numel() == n and beta.is_contiguous() and
                beta.get_device() == i and
                o.dtype is dt and o.numel() == n * d and o.is_contiguous() and o.get_device() == i and
                _is_flat(cu_seqlens, i32, N + 1, i) and
                (slot_in is None or _is_flat(slot_in, i32, N, i)) and
                (slot_out is None or _is_flat(slot_out, i32, N, i)) and
                (slot_tok is None or _is_flat(slot_tok, i32, T, i)))
    except (AttributeError, IndexError):
        good = False
    if good and T > 1:
        ldq, ldk, ldv = qs[0], ks[0], vs[0]
    else:
        if not good:
            _cache_ok(shape, cache)
            _chunk_qk(shape, q, k)
            _rows("v", v, dt, T, hv * d)
            _per_token("g", shape, g)
            _per_token("beta", shape, beta)
            _heads("o", shape, o)
            _slot_tables(shape, cache.device, cu_seqlens, slot_in, slot_out, slot_tok)
            _on(cache.device, ("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta), ("o", o))
        ldq, ldk, ldv = _row_ld(q), _row_ld(k), _row_ld(v)
    _run("gdn_recurrent_fwd", i, (
        byref(shape), q.data_ptr(), k.data_ptr(), v.data_ptr(), ldq, ldk, ldv, g.data_ptr(),
        beta.data_ptr(), scale, byref(cache), _ptr(slot_in), _ptr(slot_out), _ptr(slot_tok),
        cu_seqlens.data_ptr(), o.data_ptr(), _raw_stream(cache.device, i, stream)))


def gdn_step_fwd(shape, x, w_conv, a, b, A_log, dt_bias, z, w_norm, scale, cache, slot_in,
                 slot_out, slot_tok, cu_seqlens, out, l2_eps=1e-6, norm_eps=1e-6,
                 act=GDN_ACT_SILU, stream=None):
    """x [T, C], a, b [T, hv] and z [T, hv*d] or [T, hv, d]: rows may be
    strided.  cache: make_cache(S, conv); slot tables as gdn_recurrent_fwd."""
    i, dt, T, N, hv, d = (cache.index, _TDT[shape.dtype], shape.total_tokens, shape.n_seq, shape.hv,
                          shape.dv)
    C, f32, i32 = 2 * shape.hk * d + hv * d, torch.float32, torch.int32
    try:
        xs, as_, bs, zs = x.stride(), a.stride(), b.stride(), z.stride()
        good = (T > 0 and i >= 0 and cache.heads == (hv, d) and cache.conv_rows == (dt, C) and
                x.dtype is dt and x.shape == (T, C) and xs[1] == 1 and x.get_device() == i and
                a.dtype is dt and a.shape == (T, hv) and (as_[1] == 1 or hv == 1) and
                a.get_device() == i and
                b.dtype is dt and b.shape == (T, hv) and (bs[1] == 1 or hv == 1) and
                b.get_device() == i and
                z.dtype is dt and z.get_device() == i and
                (z.shape == (T, hv, d) and zs[2] == 1 and zs[1] == d or
                 z.shape == (T, hv * d) and zs[1] == 1) and
                w_conv.dtype is f32 and w_conv.numel() == C * 4 and w_conv.is_contiguous() and
                w_conv.get_device() == i and
                A_log.dtype is f32 and A_log.numel() == hv and A_log.is_contiguous() and
                A_log.get_device() == i and
                dt_bias.dtype is f32 and dt_bias.numel() == hv and dt_bias.is_contiguous() and
                dt_bias.get_device() == i and
                w_norm.dtype is f32 and w_norm.numel() == d and w_norm.is_contiguous() and
                w_norm.get_device() == i and
                out.dtype is dt and out.numel() == T * hv * d and out.is_contiguous() and
                out.get_device() == i and
                _is_flat(cu_seqlens, i32, N + 1, i) and
                (slot_in is None or _is_flat(slot_in, i32, N, i)) and
                (slot_out is None or slot_out is slot_in or _is_flat(slot_out, i32, N, i)) and
                (slot_tok is None or _is_flat(slot_tok, i32, T, i)))
    except (AttributeError, IndexError):
        good = False
    if good and T > 1:
        ldx, lda, ldb, ldz = xs[0], as_[0], bs[0], zs[0]
    else:
        if not good:
            if z is not None and z.dim() == 3:
                z = z.view(z.shape[0], z.shape[1] * z.shape[2])
            _cache_ok(shape, cache)
            _conv_ok(shape, x, w_conv, cu_seqlens)
            if cache.conv_rows != (dt, C):
                raise ValueError(f"the cache needs conv rows [n_slots, 3, {C}] of {dt}")
            _rows("a", a, dt, T, hv)
            _rows("b", b, dt, T, hv)
            _need("A_log", A_log, f32, hv)
            _need("dt_bias", dt_bias, f32, hv)
            _rows("z", z, dt, T, hv * d)
            _need("w_norm", w_norm, f32, d)
            _heads("out", shape, out)
            _slot_tables(shape, cache.device, cu_seqlens, slot_in, slot_out, slot_tok)
            _on(cache.device, ("x", x), ("w_conv", w_conv), ("a", a), ("b", b), ("A_log", A_log),
                ("dt_bias", dt_bias), ("z", z), ("w_norm", w_norm), ("out", out))
        ldx, lda, ldb, ldz = C if good else _row_ld(x), _row_ld(a), _row_ld(b), hv * d if good else _row_ld(z)
    _run("gdn_step_fwd", i, (
        byref(shape), x.data_ptr(), ldx, w_conv.data_ptr(), a.data_ptr(), lda, b.data_ptr(), ldb,
        A_log.data_ptr(), dt_bias.data_ptr(), z.data_ptr(), ldz, w_norm.data_ptr(), scale, l2_eps,
        norm_eps, act, byref(cache), _ptr(slot_in), _ptr(slot_out), _ptr(slot_tok),
        cu_seqlens.data_ptr(), out.data_ptr(), _raw_stream(cache.device, i, stream)))


SLOT_RANGE, SLOT_WRITTEN_TWICE, SLOT_WRITTEN_AND_READ = 1, 2, 4


def gdn_check_slots(shape, n_slots, slot_in, slot_out, slot_tok, cu_seqlens, violations,
                    stream=None):
    """Writes to violations (an int32 device tensor of one element) the bit
    mask of what is wrong with the slot tables (SLOT_*; 0 when valid)."""
    dev = cu_seqlens.device
    _slot_tables(shape, dev, cu_seqlens, slot_in, slot_out, slot_tok)
    _need("violations", violations, torch.int32, 1)
    _on(dev, ("violations", violations))
    i = cu_seqlens.get_device()
    _run("gdn_check_slots", i, (
        byref(shape), n_slots, _ptr(slot_in), _ptr(slot_out), _ptr(slot_tok), _ptr(cu_seqlens),
        _ptr(violations), _raw_stream(dev, i, stream)))


def _slot_rows(name, t):
    """[n_slots, ...] with each slot dense: (slots, bytes of a slot, bytes between slots)"""
    if t.dim() < 2 or t.shape[0] < 1 or not t[0].is_contiguous():
        raise ValueError(f"{name} must be [n_slots, ...] with each slot contiguous, got shape "
                         f"{tuple(t.shape)} strides {t.stride()}")
    size = t[0].numel() * t.element_size()
    return t.shape[0], size, t.stride(0) * t.element_size() if t.shape[0] > 1 else size


def _indexes(name, like, t, n=None):
    if t is None or not _is_flat(t, torch.int32, t.numel() if n is None else n, like.get_device()):
        _need(name, t, torch.int32, n)
        _on(like.device, (name, t))
    return t.numel()


def gdn_cache_copy(src, dst, src_idx=None, dst_idx=None, stream=None):
    """dst[dst_idx[i]] = src[src_idx[i]], whole slots of two tensors [n_slots,
    ...] of the same slot size; see libgdn.h for entries out of range."""
    n_src, size, ss = _slot_rows("src", src)
    n_dst, dsize, ds = _slot_rows("dst", dst)
    if src.dtype != dst.dtype or size != dsize:
        raise ValueError(f"slots of {size} bytes of {src.dtype} into slots of {dsize} of {dst.dtype}")
    _on(src.device, ("dst", dst))
    n = min(n_src, n_dst)
    if src_idx is not None:
        n = _indexes("src_idx", src, src_idx)
        if dst_idx is None and n > n_dst:
            raise ValueError(f"{n} slots into {n_dst}")
    if dst_idx is not None:
        n = _indexes("dst_idx", src, dst_idx, n if src_idx is not None else None)
        if src_idx is None and n > n_src:
            raise ValueError(f"{n} slots out of {n_src}")
    if src_idx is None and dst_idx is None and n_src != n_dst:
        raise ValueError(f"{n_src} slots into {n_dst} without indexes")
    i = src.get_device()
    _run("gdn_cache_copy", i, (
        _ptr(src), ss, n_src, _ptr(src_idx), _ptr(dst), ds, n_dst, _ptr(dst_idx), size, n,
        _raw_stream(src.device, i, stream)))


def gdn_cache_workspace(n_slots):
    return int(load().gdn_cache_workspace(n_slots))


class Slots:
    """A cache's buffer [n_slots, slot], counts and workspace, checked once
    and kept: what the calls below take instead of (buf, refs, ..., ws)."""

    def __init__(self, buf, refs, ws):
        if buf.dim() != 2 or not buf.is_contiguous():
            raise ValueError("the cache must be a contiguous [n_slots, slot] tensor")
        self.n_slots, self.size = buf.shape[0], buf.shape[1] * buf.element_size()
        _indexes("refs", buf, refs, self.n_slots)
        if ws is not None and not _is_flat(ws, torch.uint8, ws.numel(), buf.get_device()):
            _ws(ws)
            _on(buf.device, ("workspace", ws))
        self.buf, self.refs, self.ws = buf, refs, ws
        self.device, self.index = buf.device, buf.get_device()
        self.ptrs = _ptr(buf), _ptr(refs), _ptr(ws), 0 if ws is None else ws.numel()

    def _table(self, name, t, n=None):
        if t is None or not _is_flat(t, torch.int32, t.numel() if n is None else n, self.index):
            _need(name, t, torch.int32, n)
            _on(self.device, (name, t))
        return t.numel()

    def fork(self, src, dst, stream=None):
        n = self._table("src", src)
        self._table("dst", dst, n)
        buf, refs, ws, ws_bytes = self.ptrs
        _run("gdn_cache_fork", self.index, (
            buf, self.size, self.n_slots, refs, src.data_ptr(), n, dst.data_ptr(), ws, ws_bytes,
            _raw_stream(self.device, self.index, stream)))

    def count(self, name, slots, stream=None):
        n = self._table("slots", slots)
        _run(name, self.index, (self.ptrs[1], self.n_slots, slots.data_ptr(), n,
                                _raw_stream(self.device, self.index, stream)))

    def compact(self, remap, table, stream=None):
        self._table("remap", remap, self.n_slots)
        n = 0 if table is None else self._table("table", table)
        buf, refs, ws, ws_bytes = self.ptrs
        _run("gdn_cache_compact", self.index, (
            buf, self.size, self.n_slots, refs, remap.data_ptr(), _ptr(table), n, ws, ws_bytes,
            _raw_stream(self.device, self.index, stream)))


def gdn_cache_fork(buf, refs, src, dst, ws, stream=None):
    """Takes a free slot of buf [n_slots, slot] for every request in src and
    fills it; the slots go to dst (int32, as long as src)."""
    Slots(buf, refs, ws).fork(src, dst, stream)


def _count(name, refs, slots, stream):
    n_slots = _indexes("refs", refs, refs)
    n = _indexes("slots", refs, slots)
    i = refs.get_device()
    _run(name, i, (_ptr(refs), n_slots, _ptr(slots), n, _raw_stream(refs.device, i, stream)))


def gdn_cache_retain(refs, slots, stream=None):
    _count("gdn_cache_retain", refs, slots, stream)


def gdn_cache_release(refs, slots, stream=None):
    _count("gdn_cache_release", refs, slots, stream)


def gdn_cache_compact(buf, refs, remap, table, ws, stream=None):
    """Moves the live slots of buf to its front; remap [n_slots] receives
    where each went, and table (int32, or None) is rewritten by it."""
    Slots(buf, refs, ws).compact(remap, table, stream)
