"""Thin ctypes binding of libgdn2.so (argument marshalling only).

The ``gdn2_*`` functions mirror the C entry points of include/gdn2.h one to one:
tensor arguments may be torch tensors (their ``data_ptr()`` is passed), plain
integers (raw device addresses) or None (a null pointer).  ``chunk_fwd``,
``decode_step`` and ``chunk_bwd`` are conveniences that check shapes, allocate
the outputs and the workspace with torch on the inputs' device and raise
``Gdn2Error`` on a non-zero status.  Every step of the computation runs in the
library's CUDA kernels; there is no other code path.
"""
from __future__ import annotations

import ctypes
import functools
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libgdn2.so")

GDN2_BF16 = 0
GDN2_FP32 = 1
STATUS = {0: "GDN2_OK", -1: "GDN2_ERR_INVALID_ARG", -2: "GDN2_ERR_UNSUPPORTED", -3: "GDN2_ERR_CUDA",
          -4: "GDN2_ERR_TIMEOUT", -5: "GDN2_ERR_WORKSPACE"}

# name -> (restype, argtypes)
_P, _I, _Z, _L = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_longlong
SIGNATURES = {
    "gdn2_version": (_I, []),
    "gdn2_debug_set": (_I, [_I, ctypes.c_longlong]),
    "gdn2_status_string": (ctypes.c_char_p, [_I]),
    "gdn2_get_device_status": (_I, [_P]),
    "gdn2_chunk_fwd_workspace": (_Z, [_I] * 6),
    "gdn2_chunk_fwd": (_I, [_P] * 9 + [_I] * 6 + [_P, _Z, _P]),
    "gdn2_decode_step": (_I, [_P] * 8 + [_I] * 5 + [_P]),
    "gdn2_chunk_bwd_workspace": (_Z, [_I] * 6),
    "gdn2_chunk_bwd": (_I, [_P] * 16 + [_I] * 6 + [_P, _Z, _P]),
    "gdn2_chunk_fwd_noalloc": (_I, [_P] * 9 + [_I] * 6 + [_P]),
    "gdn2_chunk_states_bytes": (_Z, [_I] * 6),
    "gdn2_chunk_fwd_save": (_I, [_P] * 10 + [_I] * 6 + [_P, _Z, _P]),
    "gdn2_chunk_bwd_saved_workspace": (_Z, [_I] * 6),
    "gdn2_chunk_bwd_saved": (_I, [_P] * 17 + [_I] * 6 + [_P, _Z, _P]),
    "gdn2_chunk_fwd_varlen_workspace": (_Z, [_I] * 6),
    "gdn2_chunk_fwd_varlen": (_I, [_P] * 10 + [_I] * 6 + [_P, _Z, _P]),
    "gdn2_chunk_bwd_varlen_workspace": (_Z, [_I] * 6),
    "gdn2_chunk_bwd_varlen": (_I, [_P] * 17 + [_I] * 6 + [_P, _Z, _P]),
    "gdn2_chunk_states_varlen_bytes": (_Z, [_I] * 6),
    "gdn2_chunk_fwd_save_varlen": (_I, [_P] * 11 + [_I] * 6 + [_P, _Z, _P]),
    "gdn2_chunk_bwd_saved_varlen_workspace": (_Z, [_I] * 6),
    "gdn2_chunk_bwd_saved_varlen": (_I, [_P] * 18 + [_I] * 6 + [_P, _Z, _P]),
    "gdn2_chunk_fwd_kda": (_I, [_P] * 8 + [_I] * 6 + [_P, _Z, _P]),
    "gdn2_chunk_fwd_gdn": (_I, [_P] * 8 + [_I] * 6 + [_P, _Z, _P]),
    "gdn2_chunk_bwd_kda": (_I, [_P] * 14 + [_I] * 6 + [_P, _Z, _P]),
    "gdn2_chunk_bwd_gdn": (_I, [_P] * 14 + [_I] * 6 + [_P, _Z, _P]),
    "gdn2_decode_step_kda": (_I, [_P] * 7 + [_I] * 5 + [_P]),
    "gdn2_decode_step_gdn": (_I, [_P] * 7 + [_I] * 5 + [_P]),
    "gdn2_chunk_fwd_gated": (_I, [_P] * 11 + [_I] * 6 + [_P, _Z, _P]),
    "gdn2_prologue_fwd": (_I, [_P] * 6 + [_I] + [_P] * 9 + [_P] + [_I] * 6 + [_P]),
    "gdn2_prologue_bwd_workspace": (_Z, [_I] * 7),
    "gdn2_prologue_bwd": (_I, [_P] * 6 + [_I] + [_P] * 18 + [_P] + [_I] * 6 + [_P, _Z, _P]),
    "gdn2_output_gate_fwd": (_I, [_P] * 4 + [ctypes.c_longlong, _I, _I, _I, _P]),
    "gdn2_output_gate_bwd_workspace": (_Z, [ctypes.c_longlong, _I, _I]),
    "gdn2_output_gate_bwd": (_I, [_P] * 7 + [ctypes.c_longlong, _I, _I, _I, _P, _Z, _P]),
    "gdn2_ssm_fwd_workspace": (_Z, [_I] * 8),
    "gdn2_ssm_states_bytes": (_Z, [_I] * 7),
    "gdn2_ssm_fwd": (_I, [_P] * 11 + [_L] * 3 + [_I] * 7 + [_P, _Z, _P]),
    "gdn2_ssm_bwd_workspace": (_Z, [_I] * 9),
    "gdn2_ssm_bwd": (_I, [_P] * 18 + [_L] * 3 + [_I] * 7 + [_P, _Z, _P]),
    "gdn2_ssm_step": (_I, [_P] * 8 + [_L] * 3 + [_I] * 6 + [_P]),
    "gdn2_ssm_prologue_fwd": (_I, [_P] * 3 + [_I] + [_P] * 9 + [_L] * 2 + [_I] * 5 + [_P]),
    "gdn2_ssm_prologue_bwd_workspace": (_Z, [_I] * 6),
    "gdn2_ssm_prologue_bwd": (_I, [_P] * 3 + [_I] + [_P] * 15 + [_L] * 2 + [_I] * 5 + [_P, _Z, _P]),
    "gdn2_ssm_prologue_step": (_I, [_P] * 3 + [_I] + [_P] * 7 + [_L] * 2 + [_I] * 4 + [_P]),
}

_lib = None


class Gdn2Error(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__("%s failed: %s (%d)" % (what, STATUS.get(status, "unknown"), status))


def load() -> ctypes.CDLL:
    """Load the in-tree libgdn2.so.  Raises if it has not been built: there is
    no fallback implementation."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("libgdn2.so is not built (%s); run "
                              "`python -m gated_delta_rule_gdn2_b200.build`" % LIB_PATH)
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# --------------------------------------------------------------------------
# one-to-one C entry points


def gdn2_version() -> int:
    return load().gdn2_version()


GDN2_DEBUG_WAIT_LIMIT = 0
GDN2_DEBUG_WITHHOLD_READY = 1


def gdn2_debug_set(knob: int, value: int) -> int:
    return load().gdn2_debug_set(knob, value)


def gdn2_status_string(status: int) -> str:
    return load().gdn2_status_string(status).decode()


def gdn2_get_device_status(stream=None) -> int:
    return load().gdn2_get_device_status(_stream(stream))


def gdn2_chunk_fwd_workspace(B, T, H, dk, dv, dtype) -> int:
    return load().gdn2_chunk_fwd_workspace(B, T, H, dk, dv, dtype)


def gdn2_chunk_bwd_workspace(B, T, H, dk, dv, dtype) -> int:
    return load().gdn2_chunk_bwd_workspace(B, T, H, dk, dv, dtype)


def gdn2_chunk_fwd(q, k, v, log_alpha, b, w, S0, o, S_T, B, T, H, dk, dv, dtype, ws, ws_bytes,
                   stream=None) -> int:
    return load().gdn2_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w),
                                 _ptr(S0), _ptr(o), _ptr(S_T), B, T, H, dk, dv, dtype, _ptr(ws),
                                 ws_bytes, _stream(stream))


def gdn2_chunk_fwd_noalloc(q, k, v, log_alpha, b, w, S0, o, S_T, B, T, H, dk, dv, dtype,
                           stream=None) -> int:
    """gdn2_chunk_fwd for callers that cannot allocate: the scratch comes from
    a fixed 8 MiB array inside the library (see include/gdn2.h)."""
    return load().gdn2_chunk_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w),
                                         _ptr(S0), _ptr(o), _ptr(S_T), B, T, H, dk, dv, dtype,
                                         _stream(stream))


def gdn2_chunk_states_bytes(B, T, H, dk, dv, dtype) -> int:
    return load().gdn2_chunk_states_bytes(B, T, H, dk, dv, dtype)


def gdn2_chunk_bwd_saved_workspace(B, T, H, dk, dv, dtype) -> int:
    return load().gdn2_chunk_bwd_saved_workspace(B, T, H, dk, dv, dtype)


def gdn2_chunk_fwd_save(q, k, v, log_alpha, b, w, S0, o, S_T, states, B, T, H, dk, dv, dtype, ws, ws_bytes,
                        stream=None) -> int:
    return load().gdn2_chunk_fwd_save(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w),
                                      _ptr(S0), _ptr(o), _ptr(S_T), _ptr(states), B, T, H, dk, dv, dtype,
                                      _ptr(ws), ws_bytes, _stream(stream))


def gdn2_chunk_bwd_saved(q, k, v, log_alpha, b, w, S0, dO, dS_T, states, dq, dk_, dv_, dlog_alpha, db, dw,
                         dS0, B, T, H, dk, dv, dtype, ws, ws_bytes, stream=None) -> int:
    return load().gdn2_chunk_bwd_saved(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w),
                                       _ptr(S0), _ptr(dO), _ptr(dS_T), _ptr(states), _ptr(dq), _ptr(dk_),
                                       _ptr(dv_), _ptr(dlog_alpha), _ptr(db), _ptr(dw), _ptr(dS0), B, T, H,
                                       dk, dv, dtype, _ptr(ws), ws_bytes, _stream(stream))


def gdn2_decode_step(q, k, v, log_alpha, b, w, S, o, B, H, dk, dv, dtype, stream=None) -> int:
    return load().gdn2_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w),
                                   _ptr(S), _ptr(o), B, H, dk, dv, dtype, _stream(stream))


def gdn2_chunk_bwd(q, k, v, log_alpha, b, w, S0, dO, dS_T, dq, dk_, dv_, dlog_alpha, db, dw, dS0,
                   B, T, H, dk, dv, dtype, ws, ws_bytes, stream=None) -> int:
    return load().gdn2_chunk_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w),
                                 _ptr(S0), _ptr(dO), _ptr(dS_T), _ptr(dq), _ptr(dk_), _ptr(dv_),
                                 _ptr(dlog_alpha), _ptr(db), _ptr(dw), _ptr(dS0), B, T, H, dk, dv,
                                 dtype, _ptr(ws), ws_bytes, _stream(stream))


def gdn2_chunk_fwd_varlen_workspace(N, total_T, H, dk, dv, dtype) -> int:
    return load().gdn2_chunk_fwd_varlen_workspace(N, total_T, H, dk, dv, dtype)


def gdn2_chunk_fwd_varlen(q, k, v, log_alpha, b, w, S0, o, S_T, cu_seqlens, N, total_T, H, dk, dv, dtype, ws,
                          ws_bytes, stream=None) -> int:
    return load().gdn2_chunk_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w), _ptr(S0),
                                        _ptr(o), _ptr(S_T), _ptr(cu_seqlens), N, total_T, H, dk, dv, dtype,
                                        _ptr(ws), ws_bytes, _stream(stream))


def gdn2_chunk_bwd_varlen_workspace(N, total_T, H, dk, dv, dtype) -> int:
    return load().gdn2_chunk_bwd_varlen_workspace(N, total_T, H, dk, dv, dtype)


def gdn2_chunk_bwd_varlen(q, k, v, log_alpha, b, w, S0, dO, dS_T, dq, dk_, dv_, dlog_alpha, db, dw, dS0,
                          cu_seqlens, N, total_T, H, dk, dv, dtype, ws, ws_bytes, stream=None) -> int:
    return load().gdn2_chunk_bwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w), _ptr(S0),
                                        _ptr(dO), _ptr(dS_T), _ptr(dq), _ptr(dk_), _ptr(dv_), _ptr(dlog_alpha),
                                        _ptr(db), _ptr(dw), _ptr(dS0), _ptr(cu_seqlens), N, total_T, H, dk, dv,
                                        dtype, _ptr(ws), ws_bytes, _stream(stream))


def gdn2_chunk_states_varlen_bytes(N, total_T, H, dk, dv, dtype) -> int:
    return load().gdn2_chunk_states_varlen_bytes(N, total_T, H, dk, dv, dtype)


def gdn2_chunk_fwd_save_varlen(q, k, v, log_alpha, b, w, S0, o, S_T, states, cu_seqlens, N, total_T, H, dk, dv,
                               dtype, ws, ws_bytes, stream=None) -> int:
    return load().gdn2_chunk_fwd_save_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w),
                                             _ptr(S0), _ptr(o), _ptr(S_T), _ptr(states), _ptr(cu_seqlens), N,
                                             total_T, H, dk, dv, dtype, _ptr(ws), ws_bytes, _stream(stream))


def gdn2_chunk_bwd_saved_varlen_workspace(N, total_T, H, dk, dv, dtype) -> int:
    return load().gdn2_chunk_bwd_saved_varlen_workspace(N, total_T, H, dk, dv, dtype)


def gdn2_chunk_bwd_saved_varlen(q, k, v, log_alpha, b, w, S0, dO, dS_T, states, dq, dk_, dv_, dlog_alpha, db, dw,
                                dS0, cu_seqlens, N, total_T, H, dk, dv, dtype, ws, ws_bytes, stream=None) -> int:
    return load().gdn2_chunk_bwd_saved_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w),
                                              _ptr(S0), _ptr(dO), _ptr(dS_T), _ptr(states), _ptr(dq), _ptr(dk_),
                                              _ptr(dv_), _ptr(dlog_alpha), _ptr(db), _ptr(dw), _ptr(dS0),
                                              _ptr(cu_seqlens), N, total_T, H, dk, dv, dtype, _ptr(ws), ws_bytes,
                                              _stream(stream))


def _reduced(name):
    def fwd(q, k, v, log_alpha, beta, S0, o, S_T, B, T, H, dk, dv, dtype, ws, ws_bytes, stream=None):
        return getattr(load(), name)(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(S0), _ptr(o),
                                     _ptr(S_T), B, T, H, dk, dv, dtype, _ptr(ws), ws_bytes, _stream(stream))

    def bwd(q, k, v, log_alpha, beta, S0, dO, dS_T, dq, dk_, dv_, dlog_alpha, dbeta, dS0, B, T, H, dk, dv, dtype,
            ws, ws_bytes, stream=None):
        return getattr(load(), name)(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(S0), _ptr(dO),
                                     _ptr(dS_T), _ptr(dq), _ptr(dk_), _ptr(dv_), _ptr(dlog_alpha), _ptr(dbeta),
                                     _ptr(dS0), B, T, H, dk, dv, dtype, _ptr(ws), ws_bytes, _stream(stream))

    def dec(q, k, v, log_alpha, beta, S, o, B, H, dk, dv, dtype, stream=None):
        return getattr(load(), name)(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(S), _ptr(o),
                                     B, H, dk, dv, dtype, _stream(stream))

    f = {"fwd": fwd, "bwd": bwd, "dec": dec}[name.split("_")[2][:3] if "decode" not in name else "dec"]
    f.__name__ = name
    f.__doc__ = "%s of include/gdn2.h (reduced gates: one scalar beta per token and head)." % name
    return f


gdn2_chunk_fwd_kda = _reduced("gdn2_chunk_fwd_kda")
gdn2_chunk_fwd_gdn = _reduced("gdn2_chunk_fwd_gdn")
gdn2_chunk_bwd_kda = _reduced("gdn2_chunk_bwd_kda")
gdn2_chunk_bwd_gdn = _reduced("gdn2_chunk_bwd_gdn")
gdn2_decode_step_kda = _reduced("gdn2_decode_step_kda")
gdn2_decode_step_gdn = _reduced("gdn2_decode_step_gdn")


def gdn2_prologue_fwd(xq, xk, xv, Wq, Wk, Wv, K, xa, xb, xw, q, k, v, log_alpha, b, w, cu_seqlens, B, T, H, dk,
                      dv, dtype, stream=None) -> int:
    return load().gdn2_prologue_fwd(*[_ptr(t) for t in (xq, xk, xv, Wq, Wk, Wv)], K,
                                    *[_ptr(t) for t in (xa, xb, xw, q, k, v, log_alpha, b, w, cu_seqlens)],
                                    B, T, H, dk, dv, dtype, _stream(stream))


def gdn2_prologue_bwd_workspace(B, T, H, dk, dv, K, packed) -> int:
    return load().gdn2_prologue_bwd_workspace(B, T, H, dk, dv, K, int(bool(packed)))


def gdn2_prologue_bwd(xq, xk, xv, Wq, Wk, Wv, K, xa, xb, xw, dq, dk_, dv_, dlog_alpha, db, dw, dxq, dxk, dxv, dWq,
                      dWk, dWv, dxa, dxb, dxw, cu_seqlens, B, T, H, dk, dv, dtype, ws, ws_bytes, stream=None) -> int:
    return load().gdn2_prologue_bwd(*[_ptr(t) for t in (xq, xk, xv, Wq, Wk, Wv)], K,
                                    *[_ptr(t) for t in (xa, xb, xw, dq, dk_, dv_, dlog_alpha, db, dw, dxq, dxk, dxv,
                                                        dWq, dWk, dWv, dxa, dxb, dxw, cu_seqlens)],
                                    B, T, H, dk, dv, dtype, _ptr(ws), ws_bytes, _stream(stream))


def gdn2_chunk_fwd_gated(q, k, v, log_alpha, b, w, S0, g, gamma, z, S_T, B, T, H, dk, dv, dtype, ws, ws_bytes,
                         stream=None) -> int:
    return load().gdn2_chunk_fwd_gated(*[_ptr(t) for t in (q, k, v, log_alpha, b, w, S0, g, gamma, z, S_T)], B, T, H,
                                       dk, dv, dtype, _ptr(ws), ws_bytes, _stream(stream))


def gdn2_output_gate_fwd(o, g, gamma, z, rows, H, dv, dtype, stream=None) -> int:
    return load().gdn2_output_gate_fwd(_ptr(o), _ptr(g), _ptr(gamma), _ptr(z), rows, H, dv, dtype, _stream(stream))


def gdn2_output_gate_bwd_workspace(rows, H, dv) -> int:
    return load().gdn2_output_gate_bwd_workspace(rows, H, dv)


def gdn2_output_gate_bwd(o, g, gamma, dz, dO, dg, dgamma, rows, H, dv, dtype, ws, ws_bytes, stream=None) -> int:
    return load().gdn2_output_gate_bwd(_ptr(o), _ptr(g), _ptr(gamma), _ptr(dz), _ptr(dO), _ptr(dg), _ptr(dgamma),
                                       rows, H, dv, dtype, _ptr(ws), ws_bytes, _stream(stream))


def gdn2_ssm_fwd_workspace(B, T, H, G, dk, dv, dtype, packed) -> int:
    return load().gdn2_ssm_fwd_workspace(B, T, H, G, dk, dv, dtype, int(bool(packed)))


def gdn2_ssm_states_bytes(B, T, H, dk, dv, dtype, packed) -> int:
    return load().gdn2_ssm_states_bytes(B, T, H, dk, dv, dtype, int(bool(packed)))


def gdn2_ssm_fwd(q, k, v, log_alpha, dt, skip, S0, o, S_T, states, cu_seqlens, ldq, ldk, ldv, B, T, H, G, dk, dv,
                 dtype, ws, ws_bytes, stream=None) -> int:
    return load().gdn2_ssm_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(dt), _ptr(skip), _ptr(S0), _ptr(o),
                               _ptr(S_T), _ptr(states), _ptr(cu_seqlens), ldq, ldk, ldv, B, T, H, G, dk, dv, dtype,
                               _ptr(ws), ws_bytes, _stream(stream))


def gdn2_ssm_bwd_workspace(B, T, H, G, dk, dv, dtype, packed, states_given) -> int:
    return load().gdn2_ssm_bwd_workspace(B, T, H, G, dk, dv, dtype, int(bool(packed)), int(bool(states_given)))


def gdn2_ssm_bwd(q, k, v, log_alpha, dt, skip, S0, dO, dS_T, states, dq, dk_, dv_, dlog_alpha, ddt, dskip, dS0,
                 cu_seqlens, ldq, ldk, ldv, B, T, H, G, dk, dv, dtype, ws, ws_bytes, stream=None) -> int:
    return load().gdn2_ssm_bwd(*map(_ptr, (q, k, v, log_alpha, dt, skip, S0, dO, dS_T, states, dq, dk_, dv_,
                                           dlog_alpha, ddt, dskip, dS0, cu_seqlens)),
                               ldq, ldk, ldv, B, T, H, G, dk, dv, dtype, _ptr(ws), ws_bytes, _stream(stream))


def gdn2_ssm_step(q, k, v, log_alpha, dt, skip, S, o, ldq, ldk, ldv, B, H, G, dk, dv, dtype, stream=None) -> int:
    return load().gdn2_ssm_step(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(dt), _ptr(skip), _ptr(S), _ptr(o),
                                ldq, ldk, ldv, B, H, G, dk, dv, dtype, _stream(stream))


def gdn2_ssm_prologue_fwd(x, W, bias, K, xdt, dt_bias, A_log, init, y, dt, log_alpha, window, cu_seqlens, ldx, ldt,
                          B, T, C, H, dtype, stream=None) -> int:
    return load().gdn2_ssm_prologue_fwd(_ptr(x), _ptr(W), _ptr(bias), K,
                                        *map(_ptr, (xdt, dt_bias, A_log, init, y, dt, log_alpha, window, cu_seqlens)),
                                        ldx, ldt, B, T, C, H, dtype, _stream(stream))


def gdn2_ssm_prologue_bwd_workspace(B, T, C, K, H, packed) -> int:
    return load().gdn2_ssm_prologue_bwd_workspace(B, T, C, K, H, int(bool(packed)))


def gdn2_ssm_prologue_bwd(x, W, bias, K, xdt, dt_bias, A_log, init, dy, ddt, dlog_alpha, dx, dW, dbias, dxdt,
                          ddt_bias, dA_log, dinit, cu_seqlens, ldx, ldt, B, T, C, H, dtype, ws, ws_bytes,
                          stream=None) -> int:
    return load().gdn2_ssm_prologue_bwd(_ptr(x), _ptr(W), _ptr(bias), K,
                                        *map(_ptr, (xdt, dt_bias, A_log, init, dy, ddt, dlog_alpha, dx, dW, dbias, dxdt,
                                                    ddt_bias, dA_log, dinit, cu_seqlens)),
                                        ldx, ldt, B, T, C, H, dtype, _ptr(ws), ws_bytes, _stream(stream))


def gdn2_ssm_prologue_step(x, W, bias, K, xdt, dt_bias, A_log, window, y, dt, log_alpha, ldx, ldt, B, C, H, dtype,
                           stream=None) -> int:
    return load().gdn2_ssm_prologue_step(_ptr(x), _ptr(W), _ptr(bias), K,
                                         *map(_ptr, (xdt, dt_bias, A_log, window, y, dt, log_alpha)), ldx, ldt, B, C, H,
                                         dtype, _stream(stream))


# --------------------------------------------------------------------------
# torch conveniences
#
# stream= (a torch stream or a raw handle): the call runs, and allocates what it
# returns, as if that stream were the current one.  The caller orders it behind
# the making of its inputs, keeps these alive until it has run, and orders what
# reads its outputs on another stream behind it.


def _there(fn, t, stream, *args, **kw):
    """fn(*args, **kw) with t's device current and, where one is given, `stream`
    (a torch stream or a handle) as its current stream.  What the call allocates
    then comes from that stream's own memory pool: a block of the calling
    stream's pool may still be in use by work that stream has pending, and
    nothing orders the call behind it."""
    import torch
    with torch.cuda.device(t.device):
        if stream is None:
            return fn(*args, **kw)
        if isinstance(stream, int):
            # (a handle of 0 is the default stream; torch would make a stream of its own of it)
            stream = torch.cuda.ExternalStream(stream, device=t.device) if stream else torch.cuda.default_stream(t.device)
        if stream.device != t.device:
            raise ValueError("stream is on %s, the tensors on %s" % (stream.device, t.device))
        with torch.cuda.stream(stream):
            return fn(*args, **kw)


def _on_stream(fn):
    """fn, whose last argument is `stream`, called with that stream current where one is given."""
    at = fn.__code__.co_argcount - 1
    first = fn.__code__.co_varnames[0]

    @functools.wraps(fn)
    def call(*args, **kw):
        stream = kw.pop("stream", None) if len(args) <= at else args[at]
        if stream is None:
            return fn(*args, **kw)
        return _there(fn, args[0] if args else kw[first], stream, *args[:at], **kw)

    return call


def _dtype_code(t):
    import torch
    if t.dtype == torch.bfloat16:
        return GDN2_BF16
    if t.dtype == torch.float32:
        return GDN2_FP32
    raise TypeError("token tensors must be bfloat16 or float32, got %s" % t.dtype)


def _check_tokens(q, k, v, log_alpha, b, w, lead_dims):
    dt = q.dtype
    for name, t in (("q", q), ("k", k), ("v", v), ("log_alpha", log_alpha), ("b", b), ("w", w)):
        if not t.is_cuda or not t.is_contiguous() or t.dtype != dt:
            raise ValueError("%s must be a contiguous CUDA tensor of dtype %s" % (name, dt))
    lead = tuple(q.shape[:lead_dims])
    for t in (k, log_alpha, b):
        if tuple(t.shape) != tuple(q.shape):
            raise ValueError("q, k, log_alpha and b must share a shape")
    if tuple(w.shape) != tuple(v.shape) or tuple(v.shape[:lead_dims]) != lead:
        raise ValueError("v and w must be %s + (dv,)" % (lead,))


def _raise(st, what):
    if st != 0:
        raise Gdn2Error(st, what)


@_on_stream
def chunk_fwd(q, k, v, log_alpha, b, w, S0=None, output_final_state=True, save_states=False, stream=None):
    """o, S_T = chunk_fwd(...) for token tensors [B,T,H,D] (bf16 or fp32).

    With save_states=True returns (o, S_T, states): the chunk-boundary states
    for chunk_bwd(..., states=states)."""
    import torch
    _check_tokens(q, k, v, log_alpha, b, w, 3)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    o = torch.empty((B, T, H, dv), dtype=q.dtype, device=q.device)
    S_T = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device) if output_final_state else None
    nws = gdn2_chunk_fwd_workspace(B, T, H, dk, dv, dt)
    ws = torch.empty(nws, dtype=torch.uint8, device=q.device) if nws else None
    if not save_states:
        _raise(gdn2_chunk_fwd(q, k, v, log_alpha, b, w, S0, o, S_T, B, T, H, dk, dv, dt, ws, nws, stream),
               "gdn2_chunk_fwd")
        return o, S_T
    nst = gdn2_chunk_states_bytes(B, T, H, dk, dv, dt)
    states = torch.empty(nst, dtype=torch.uint8, device=q.device) if nst else None
    _raise(gdn2_chunk_fwd_save(q, k, v, log_alpha, b, w, S0, o, S_T, states, B, T, H, dk, dv, dt, ws, nws,
                               stream), "gdn2_chunk_fwd_save")
    return o, S_T, states


@_on_stream
def decode_step(q, k, v, log_alpha, b, w, S, stream=None):
    """o = decode_step(...): tokens [B,H,D]; S [B,H,dk,dv] fp32 updated in place."""
    import torch
    _check_tokens(q, k, v, log_alpha, b, w, 2)
    B, H, dk = q.shape
    dv = v.shape[-1]
    if S.dtype != torch.float32 or tuple(S.shape) != (B, H, dk, dv) or not S.is_contiguous():
        raise ValueError("S must be a contiguous fp32 tensor of shape %s" % ((B, H, dk, dv),))
    o = torch.empty((B, H, dv), dtype=q.dtype, device=q.device)
    _raise(gdn2_decode_step(q, k, v, log_alpha, b, w, S, o, B, H, dk, dv, _dtype_code(q), stream),
           "gdn2_decode_step")
    return o


@_on_stream
def chunk_bwd(q, k, v, log_alpha, b, w, S0, dO, dS_T=None, need_dS0=True, states=None, stream=None):
    """Gradients (dq, dk, dv, dlog_alpha, db, dw, dS0) of gdn2_chunk_fwd.

    `states` from chunk_fwd(..., save_states=True) skips the state recompute."""
    import torch
    _check_tokens(q, k, v, log_alpha, b, w, 3)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    g = {n: torch.empty_like(q) for n in ("dq", "dk", "dlog_alpha", "db")}
    g.update({n: torch.empty_like(v) for n in ("dv", "dw")})
    g["dS0"] = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device) if need_dS0 else None
    if states is None:
        nws = gdn2_chunk_bwd_workspace(B, T, H, dk, dv, dt)
        ws = torch.empty(nws, dtype=torch.uint8, device=q.device) if nws else None
        _raise(gdn2_chunk_bwd(q, k, v, log_alpha, b, w, S0, dO, dS_T, g["dq"], g["dk"], g["dv"],
                              g["dlog_alpha"], g["db"], g["dw"], g["dS0"], B, T, H, dk, dv, dt, ws, nws,
                              stream), "gdn2_chunk_bwd")
        return g
    nws = gdn2_chunk_bwd_saved_workspace(B, T, H, dk, dv, dt)
    ws = torch.empty(nws, dtype=torch.uint8, device=q.device) if nws else None
    _raise(gdn2_chunk_bwd_saved(q, k, v, log_alpha, b, w, S0, dO, dS_T, states, g["dq"], g["dk"], g["dv"],
                                g["dlog_alpha"], g["db"], g["dw"], g["dS0"], B, T, H, dk, dv, dt, ws, nws,
                                stream), "gdn2_chunk_bwd_saved")
    return g


def _check_cu(cu_seqlens, total_T):
    import torch
    if not cu_seqlens.is_cuda or cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or \
            not cu_seqlens.is_contiguous() or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be a contiguous 1-D int32 CUDA tensor of N + 1 offsets")
    return cu_seqlens.numel() - 1


@_on_stream
def chunk_fwd_varlen(q, k, v, log_alpha, b, w, cu_seqlens, S0=None, output_final_state=True, save_states=False,
                     stream=None):
    """o, S_T = chunk_fwd_varlen(...) for packed token tensors [total_T, H, D]
    (or [1, total_T, H, D]) holding N sequences delimited by cu_seqlens (N + 1
    int32 offsets on the device).  S0 / S_T are [N, H, dk, dv].  With
    save_states=True returns (o, S_T, states) for chunk_bwd_varlen."""
    import torch
    q, k, v, log_alpha, b, w = (t.reshape(t.shape[-3:]) if t.dim() == 4 else t for t in (q, k, v, log_alpha, b, w))
    _check_tokens(q, k, v, log_alpha, b, w, 2)
    T, H, dk = q.shape
    dv = v.shape[-1]
    N = _check_cu(cu_seqlens, T)
    dt = _dtype_code(q)
    o = torch.empty((T, H, dv), dtype=q.dtype, device=q.device)
    S_T = torch.empty((N, H, dk, dv), dtype=torch.float32, device=q.device) if output_final_state else None
    nws = gdn2_chunk_fwd_varlen_workspace(N, T, H, dk, dv, dt)
    ws = torch.empty(nws, dtype=torch.uint8, device=q.device) if nws else None
    if not save_states:
        _raise(gdn2_chunk_fwd_varlen(q, k, v, log_alpha, b, w, S0, o, S_T, cu_seqlens, N, T, H, dk, dv, dt, ws, nws,
                                     stream), "gdn2_chunk_fwd_varlen")
        return o, S_T
    nst = gdn2_chunk_states_varlen_bytes(N, T, H, dk, dv, dt)
    states = torch.empty(nst, dtype=torch.uint8, device=q.device) if nst else None
    _raise(gdn2_chunk_fwd_save_varlen(q, k, v, log_alpha, b, w, S0, o, S_T, states, cu_seqlens, N, T, H, dk, dv, dt,
                                      ws, nws, stream), "gdn2_chunk_fwd_save_varlen")
    return o, S_T, states


@_on_stream
def chunk_bwd_varlen(q, k, v, log_alpha, b, w, cu_seqlens, S0, dO, dS_T=None, need_dS0=True, states=None,
                     stream=None):
    """Gradients of chunk_fwd_varlen: dq, dk, dv, dlog_alpha, db, dw as [total_T, H, D], dS0 [N, H, dk, dv]."""
    import torch
    q, k, v, log_alpha, b, w, dO = (t.reshape(t.shape[-3:]) if t.dim() == 4 else t
                                    for t in (q, k, v, log_alpha, b, w, dO))
    _check_tokens(q, k, v, log_alpha, b, w, 2)
    T, H, dk = q.shape
    dv = v.shape[-1]
    N = _check_cu(cu_seqlens, T)
    dt = _dtype_code(q)
    g = {n: torch.empty_like(q) for n in ("dq", "dk", "dlog_alpha", "db")}
    g.update({n: torch.empty_like(v) for n in ("dv", "dw")})
    g["dS0"] = torch.empty((N, H, dk, dv), dtype=torch.float32, device=q.device) if need_dS0 else None
    if states is None:
        nws = gdn2_chunk_bwd_varlen_workspace(N, T, H, dk, dv, dt)
        ws = torch.empty(nws, dtype=torch.uint8, device=q.device) if nws else None
        _raise(gdn2_chunk_bwd_varlen(q, k, v, log_alpha, b, w, S0, dO, dS_T, g["dq"], g["dk"], g["dv"],
                                     g["dlog_alpha"], g["db"], g["dw"], g["dS0"], cu_seqlens, N, T, H, dk, dv, dt,
                                     ws, nws, stream), "gdn2_chunk_bwd_varlen")
        return g
    nws = gdn2_chunk_bwd_saved_varlen_workspace(N, T, H, dk, dv, dt)
    ws = torch.empty(nws, dtype=torch.uint8, device=q.device) if nws else None
    _raise(gdn2_chunk_bwd_saved_varlen(q, k, v, log_alpha, b, w, S0, dO, dS_T, states, g["dq"], g["dk"], g["dv"],
                                       g["dlog_alpha"], g["db"], g["dw"], g["dS0"], cu_seqlens, N, T, H, dk, dv,
                                       dt, ws, nws, stream), "gdn2_chunk_bwd_saved_varlen")
    return g


def _check_reduced(q, k, v, log_alpha, beta, mode, lead_dims):
    if mode not in ("kda", "gdn"):
        raise ValueError("mode must be 'kda' or 'gdn'")
    lead = tuple(q.shape[:lead_dims])
    for name, t in (("q", q), ("k", k), ("v", v), ("log_alpha", log_alpha), ("beta", beta)):
        if not t.is_cuda or not t.is_contiguous() or t.dtype != q.dtype:
            raise ValueError("%s must be a contiguous CUDA tensor of dtype %s" % (name, q.dtype))
    want_la = q.shape if mode == "kda" else lead
    if tuple(k.shape) != tuple(q.shape) or tuple(log_alpha.shape) != tuple(want_la) or tuple(beta.shape) != lead \
            or tuple(v.shape[:lead_dims]) != lead:
        raise ValueError("shapes: q, k %s; log_alpha %s; beta %s" % (tuple(q.shape), tuple(want_la), lead))


@_on_stream
def chunk_fwd_reduced(q, k, v, log_alpha, beta, mode="kda", S0=None, output_final_state=True, stream=None):
    """o, S_T with reduced gates: mode 'kda' (beta [B,T,H] for both gates,
    log_alpha [B,T,H,dk]) or 'gdn' (also a scalar decay, log_alpha [B,T,H])."""
    import torch
    _check_reduced(q, k, v, log_alpha, beta, mode, 3)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    o = torch.empty((B, T, H, dv), dtype=q.dtype, device=q.device)
    S_T = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device) if output_final_state else None
    nws = gdn2_chunk_fwd_workspace(B, T, H, dk, dv, dt)
    ws = torch.empty(nws, dtype=torch.uint8, device=q.device) if nws else None
    fn = gdn2_chunk_fwd_kda if mode == "kda" else gdn2_chunk_fwd_gdn
    _raise(fn(q, k, v, log_alpha, beta, S0, o, S_T, B, T, H, dk, dv, dt, ws, nws, stream), fn.__name__)
    return o, S_T


@_on_stream
def chunk_bwd_reduced(q, k, v, log_alpha, beta, S0, dO, dS_T=None, mode="kda", need_dS0=True, stream=None):
    """Gradients with reduced gates: dq, dk, dv, dlog_alpha (the shape of
    log_alpha), dbeta [B,T,H] and dS0."""
    import torch
    _check_reduced(q, k, v, log_alpha, beta, mode, 3)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    g = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v),
         "dlog_alpha": torch.empty_like(log_alpha), "dbeta": torch.empty_like(beta),
         "dS0": torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device) if need_dS0 else None}
    nws = gdn2_chunk_bwd_workspace(B, T, H, dk, dv, dt)
    ws = torch.empty(nws, dtype=torch.uint8, device=q.device) if nws else None
    fn = gdn2_chunk_bwd_kda if mode == "kda" else gdn2_chunk_bwd_gdn
    _raise(fn(q, k, v, log_alpha, beta, S0, dO, dS_T, g["dq"], g["dk"], g["dv"], g["dlog_alpha"], g["dbeta"],
              g["dS0"], B, T, H, dk, dv, dt, ws, nws, stream), fn.__name__)
    return g


@_on_stream
def decode_step_reduced(q, k, v, log_alpha, beta, S, mode="kda", stream=None):
    """o = one decode step with reduced gates (beta [B,H]; 'gdn': log_alpha [B,H]); S updated in place."""
    import torch
    _check_reduced(q, k, v, log_alpha, beta, mode, 2)
    B, H, dk = q.shape
    dv = v.shape[-1]
    o = torch.empty((B, H, dv), dtype=q.dtype, device=q.device)
    fn = gdn2_decode_step_kda if mode == "kda" else gdn2_decode_step_gdn
    _raise(fn(q, k, v, log_alpha, beta, S, o, B, H, dk, dv, _dtype_code(q), stream), fn.__name__)
    return o


@_on_stream
def prologue(xq, xk, xv, Wq, Wk, Wv, xa, xb, xw, cu_seqlens=None, stream=None):
    """The mixer's inputs (q, k, v, log_alpha, b, w) from the projections and
    gate pre-activations: token tensors [B, T, H, D] (or packed [T, H, D] with
    cu_seqlens), filters fp32 [H*D, K]."""
    import torch
    packed = cu_seqlens is not None
    H, dk = xq.shape[-2], xq.shape[-1]
    dv = xv.shape[-1]
    B, T = (cu_seqlens.numel() - 1, xq.shape[0]) if packed else (xq.shape[0], xq.shape[1])
    K = Wq.shape[-1]
    outs = [torch.empty_like(t) for t in (xq, xk, xv, xa, xb, xw)]
    _raise(gdn2_prologue_fwd(xq, xk, xv, Wq, Wk, Wv, K, xa, xb, xw, *outs, cu_seqlens, B, T, H, dk, dv,
                             _dtype_code(xq), stream), "gdn2_prologue_fwd")
    return dict(zip(("q", "k", "v", "log_alpha", "b", "w"), outs))


@_on_stream
def prologue_bwd(xq, xk, xv, Wq, Wk, Wv, xa, xb, xw, grads, cu_seqlens=None, stream=None):
    """Gradients of the prologue's inputs from `grads` (dq, dk, dv, dlog_alpha, db, dw)."""
    import torch
    packed = cu_seqlens is not None
    H, dk = xq.shape[-2], xq.shape[-1]
    dv = xv.shape[-1]
    B, T = (cu_seqlens.numel() - 1, xq.shape[0]) if packed else (xq.shape[0], xq.shape[1])
    K = Wq.shape[-1]
    dx = {n: torch.empty_like(t) for n, t in (("dxq", xq), ("dxk", xk), ("dxv", xv), ("dxa", xa), ("dxb", xb),
                                             ("dxw", xw))}
    dW = {n: torch.empty_like(t) for n, t in (("dWq", Wq), ("dWk", Wk), ("dWv", Wv))}
    nws = gdn2_prologue_bwd_workspace(B, T, H, dk, dv, K, packed)
    ws = torch.empty(max(nws, 16), dtype=torch.uint8, device=xq.device)
    _raise(gdn2_prologue_bwd(xq, xk, xv, Wq, Wk, Wv, K, xa, xb, xw, grads["dq"], grads["dk"], grads["dv"],
                             grads["dlog_alpha"], grads["db"], grads["dw"], dx["dxq"], dx["dxk"], dx["dxv"],
                             dW["dWq"], dW["dWk"], dW["dWv"], dx["dxa"], dx["dxb"], dx["dxw"], cu_seqlens, B, T, H,
                             dk, dv, _dtype_code(xq), ws, nws, stream), "gdn2_prologue_bwd")
    dx.update(dW)
    return dx


@_on_stream
def output_gate(o, g, gamma, stream=None):
    """z = o / rms(o) * gamma * silu(g) per token and head (o, g [..., H, dv], gamma fp32 [dv])."""
    import torch
    H, dv = o.shape[-2], o.shape[-1]
    rows = o.numel() // (H * dv)
    z = torch.empty_like(o)
    _raise(gdn2_output_gate_fwd(o, g, gamma, z, rows, H, dv, _dtype_code(o), stream), "gdn2_output_gate_fwd")
    return z


@_on_stream
def output_gate_bwd(o, g, gamma, dz, stream=None):
    """(do, dg, dgamma) of output_gate."""
    import torch
    H, dv = o.shape[-2], o.shape[-1]
    rows = o.numel() // (H * dv)
    dO, dg, dgamma = torch.empty_like(o), torch.empty_like(g), torch.empty_like(gamma)
    nws = gdn2_output_gate_bwd_workspace(rows, H, dv)
    ws = torch.empty(max(nws, 16), dtype=torch.uint8, device=o.device)
    _raise(gdn2_output_gate_bwd(o, g, gamma, dz, dO, dg, dgamma, rows, H, dv, _dtype_code(o), ws, nws, stream),
           "gdn2_output_gate_bwd")
    return dO, dg, dgamma


@_on_stream
def chunk_fwd_gated(q, k, v, log_alpha, b, w, g, gamma, S0=None, output_final_state=True, stream=None):
    """z, S_T: the forward with the output epilogue z = o / rms(o) * gamma * silu(g)."""
    import torch
    _check_tokens(q, k, v, log_alpha, b, w, 3)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    z = torch.empty((B, T, H, dv), dtype=q.dtype, device=q.device)
    S_T = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device) if output_final_state else None
    nws = gdn2_chunk_fwd_workspace(B, T, H, dk, dv, dt)
    ws = torch.empty(nws, dtype=torch.uint8, device=q.device) if nws else None
    _raise(gdn2_chunk_fwd_gated(q, k, v, log_alpha, b, w, S0, g, gamma, z, S_T, B, T, H, dk, dv, dt, ws, nws,
                                stream), "gdn2_chunk_fwd_gated")
    return z, S_T


# --------------------------------------------------------------------------
# selective state space scan and its prologue
#
# A single token's call is over in microseconds, so these checks are written to
# cost little: shapes and strides are read once, and contiguous tensors take a
# short way.


def _elsewhere(t):
    """Whether t's device is not the current one (the call is then made again
    with it current: workspace sizes and launches go by the current device)."""
    import torch
    i = t.get_device()
    if i < 0:
        raise ValueError("tensors must be CUDA tensors, got one on %s" % t.device)
    return i != torch._C._cuda_getDevice()


def _raw_stream(t):
    import torch
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _scratch(n, like):
    """n bytes of workspace on like's device (None for none), of the current stream's pool."""
    import torch
    return like.new_empty(n, dtype=torch.uint8) if n else None


def _at(t):
    return None if t is None else t.data_ptr()


def _row_ld(name, t, n, width):
    """Elements between the rows of t, whose inner dimensions are contiguous
    and whose n leading ones are rows at one distance."""
    if t.is_contiguous():
        return width
    st, sh = t.stride(), t.shape
    if st[-1] == 1 and (len(st) == n + 1 or st[-2] == sh[-1]):  # slices of wider rows, in few steps
        if n == 1 and sh[0] > 1:
            return st[0]
        if n == 2 and sh[1] > 1 and (sh[0] == 1 or st[0] == st[1] * sh[1]):
            return st[1]
    step = 1
    for d in range(t.dim() - 1, n - 1, -1):
        if sh[d] != 1 and st[d] != step:
            raise ValueError("%s must be contiguous within a row" % name)
        step *= sh[d]
    ld, rows = None, 1  # the distance is that of the last leading dimension longer than one
    for d in range(n - 1, -1, -1):
        if sh[d] != 1:
            if ld is None:
                ld = st[d]
            elif st[d] != ld * rows:
                raise ValueError("%s must have its rows at one distance" % name)
        rows *= sh[d]
    return width if ld is None else ld


def _check_like(name, t, shape, dtype, dev):
    """A contiguous tensor of this shape and dtype on device number dev."""
    if t.shape != shape or t.dtype != dtype or t.get_device() != dev or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of shape %s on cuda:%d" % (name, dtype, tuple(shape), dev))


def _check_f32(name, t, shape, dev):
    import torch
    _check_like(name, t, shape, torch.float32, dev)


def _empty_as(t):
    """An empty contiguous tensor of t's shape, dtype and device (empty_like
    takes half the time of new_empty with a shape)."""
    import torch
    return torch.empty_like(t) if t.is_contiguous() else torch.empty_like(t, memory_format=torch.contiguous_format)


def _scan_sizes(q, k, v, log_alpha, dt, skip, cu_seqlens, lead_dims):
    if cu_seqlens is not None:
        lead_dims = 1
    vs, qs, dtype, dev = v.shape, q.shape, q.dtype, q.get_device()
    if len(vs) != lead_dims + 2 or len(qs) != lead_dims + 2:
        raise ValueError("v must be %s + (H, dv) and q, k (G, dk)" % ("[rows]" if lead_dims == 1 else "[B, T]"))
    H, dv, G, dk = vs[-2], vs[-1], qs[-2], qs[-1]
    if k.shape != qs or G < 1 or H % G:
        raise ValueError("q and k must share a shape [.., G, dk], G dividing H = %d" % H)
    if k.dtype != dtype or v.dtype != dtype or k.get_device() != dev or v.get_device() != dev:
        raise ValueError("q, k and v must be of one dtype and on one device")
    hs = vs[:-1]
    lead = hs[:-1]
    if qs[:-2] != lead:
        raise ValueError("q must have leading dimensions %s, got %s" % (tuple(lead), tuple(qs)))
    ldq = G * dk if q.is_contiguous() else _row_ld("q", q, lead_dims, G * dk)
    ldk = G * dk if k.is_contiguous() else _row_ld("k", k, lead_dims, G * dk)
    ldv = H * dv if v.is_contiguous() else _row_ld("v", v, lead_dims, H * dv)
    _check_like("log_alpha", log_alpha, hs, dtype, dev)
    _check_like("dt", dt, hs, dtype, dev)
    if skip is not None:
        _check_f32("skip", skip, (H,), dev)
    if cu_seqlens is None:
        B, T = (vs[0], 1) if lead_dims == 1 else lead
    else:
        B, T = _check_cu(cu_seqlens, vs[0]), vs[0]
        if cu_seqlens.get_device() != dev:
            raise ValueError("cu_seqlens must be on %s" % q.device)
    return hs, dev, B, T, H, G, dk, dv, ldq, ldk, ldv


def _like_rows(ts, lds):
    """Empty tensors with the shapes and row distances of ts.  Those that are
    separate slices of one tensor's rows become slices of one tensor again: each
    with rows of its own, as far apart, would take that tensor's size."""
    out, groups = [None] * len(ts), {}
    for i, (t, ld) in enumerate(zip(ts, lds)):
        if ld == t.shape[-2] * t.shape[-1]:
            out[i] = _empty_as(t)
        else:
            groups.setdefault((t.untyped_storage().data_ptr(), ld), []).append(i)
    for (_, ld), g in groups.items():
        g.sort(key=lambda i: ts[i].storage_offset())
        at = [ts[i].storage_offset() for i in g]
        end = [a + ts[i].shape[-2] * ts[i].shape[-1] for a, i in zip(at, g)]
        if len(g) == 1 or end[-1] - at[0] > ld or any(e > a for e, a in zip(end, at[1:])):
            for i in g:
                out[i] = ts[i].new_empty_strided(ts[i].shape, ts[i].stride())
            continue
        t = ts[g[0]]
        rows = t.numel() // (t.shape[-2] * t.shape[-1])
        both = t.new_empty((rows - 1) * ld + end[-1] - at[0])
        for i, a in zip(g, at):
            out[i] = both.as_strided(ts[i].shape, ts[i].stride(), a - at[0])
    return out


def ssm_fwd(q, k, v, log_alpha, dt, skip=None, S0=None, output_final_state=True, save_states=False, cu_seqlens=None,
            stream=None):
    """o, S_T of the selective state space scan S_t = e^{log_alpha_t} S_{t-1} +
    dt_t k_t v_t^T, o_t = S_t^T q_t + skip v_t.

    v [B, T, H, dv]; q, k [B, T, G, dk], each group read by H / G heads;
    log_alpha <= 0 and dt >= 0 [B, T, H]; skip fp32 [H]; S0 fp32 [B, H, dk, dv].
    q, k, v may be views with a longer row stride.  Packed: [rows, ..] tensors
    and cu_seqlens (B + 1 int32 offsets on the device).  With save_states=True
    returns (o, S_T, states) for ssm_bwd(..., states=states)."""
    if _elsewhere(q) or stream is not None:
        return _there(ssm_fwd, q, stream, q, k, v, log_alpha, dt, skip, S0, output_final_state, save_states, cu_seqlens)
    import torch
    _, dev, B, T, H, G, dk, dv, ldq, ldk, ldv = _scan_sizes(q, k, v, log_alpha, dt, skip, cu_seqlens, 2)
    code, packed = _dtype_code(q), cu_seqlens is not None
    if S0 is not None:
        _check_f32("S0", S0, (B, H, dk, dv), dev)
    o, S_T = _empty_as(v), None
    if output_final_state:
        S_T = v.new_empty((B, H, dk, dv), dtype=torch.float32) if S0 is None else torch.empty_like(S0)
    states = None
    if save_states:
        states = v.new_empty(gdn2_ssm_states_bytes(B, T, H, dk, dv, code, packed), dtype=torch.uint8)
    nws = load().gdn2_ssm_fwd_workspace(B, T, H, G, dk, dv, code, packed)
    ws = _scratch(nws, q)
    _raise(load().gdn2_ssm_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_alpha.data_ptr(), dt.data_ptr(), _at(skip),
                               _at(S0), o.data_ptr(), _at(S_T), _at(states), _at(cu_seqlens), ldq, ldk, ldv, B, T, H, G,
                               dk, dv, code, _at(ws), nws, _raw_stream(q)), "gdn2_ssm_fwd")
    return (o, S_T, states) if save_states else (o, S_T)


def ssm_bwd(q, k, v, log_alpha, dt, dO, skip=None, S0=None, dS_T=None, states=None, need_dS0=True, cu_seqlens=None,
            into=None, stream=None):
    """Gradients (dq, dk, dv, dlog_alpha, ddt, dskip, dS0) of ssm_fwd from dO
    and dS_T.  `states` from ssm_fwd(..., save_states=True) on the same inputs
    skips forming them anew.  dq, dk, dv have their input's strides (slices of
    one tensor's rows: as slices of one new tensor); `into`
    (dq, dk, dv) gives the tensors to write them to, such as views of the
    prologue's dy, which may not overlap one another."""
    if _elsewhere(q) or stream is not None:
        return _there(ssm_bwd, q, stream, q, k, v, log_alpha, dt, dO, skip, S0, dS_T, states, need_dS0, cu_seqlens, into)
    import torch
    hs, dev, B, T, H, G, dk, dv, ldq, ldk, ldv = _scan_sizes(q, k, v, log_alpha, dt, skip, cu_seqlens, 2)
    code, packed = _dtype_code(q), cu_seqlens is not None
    for name, t in (("S0", S0), ("dS_T", dS_T)):
        if t is not None:
            _check_f32(name, t, (B, H, dk, dv), dev)
    _check_like("dO", dO, v.shape, q.dtype, dev)
    if states is not None and (states.dtype != torch.uint8 or states.get_device() != dev or
                               not states.is_contiguous() or
                               states.numel() != gdn2_ssm_states_bytes(B, T, H, dk, dv, code, packed)):
        raise ValueError("states must be what ssm_fwd(..., save_states=True) returned for these sizes")
    for name, t, x, ld, w in zip(("dq", "dk", "dv"), into or (), (q, k, v), (ldq, ldk, ldv), (G * dk, G * dk, H * dv)):
        if t.shape != x.shape or t.dtype != x.dtype or t.get_device() != dev or _row_ld(name, t, len(hs) - 1, w) != ld:
            raise ValueError("%s must have its input's shape, dtype and row stride" % name)
    dq, dk_, dv_ = into or _like_rows((q, k, v), (ldq, ldk, ldv))
    g = {"dq": dq, "dk": dk_, "dv": dv_, "dlog_alpha": torch.empty_like(log_alpha), "ddt": torch.empty_like(dt),
         "dskip": None if skip is None else torch.empty_like(skip),
         "dS0": None}
    if need_dS0:
        like = S0 if S0 is not None else dS_T
        g["dS0"] = q.new_empty((B, H, dk, dv), dtype=torch.float32) if like is None else torch.empty_like(like)
    nws = load().gdn2_ssm_bwd_workspace(B, T, H, G, dk, dv, code, packed, states is not None)
    ws = _scratch(nws, q)
    _raise(load().gdn2_ssm_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_alpha.data_ptr(), dt.data_ptr(), _at(skip),
                               _at(S0), dO.data_ptr(), _at(dS_T), _at(states), dq.data_ptr(), dk_.data_ptr(),
                               dv_.data_ptr(), g["dlog_alpha"].data_ptr(), g["ddt"].data_ptr(), _at(g["dskip"]),
                               _at(g["dS0"]), _at(cu_seqlens), ldq, ldk, ldv, B, T, H, G, dk, dv, code, _at(ws), nws,
                               _raw_stream(q)), "gdn2_ssm_bwd")
    return g


def ssm_step(q, k, v, log_alpha, dt, S, skip=None, stream=None):
    """o = one token of the scan: v [B, H, dv], q, k [B, G, dk], log_alpha, dt
    [B, H]; S fp32 [B, H, dk, dv] updated in place."""
    if _elsewhere(q) or stream is not None:
        return _there(ssm_step, q, stream, q, k, v, log_alpha, dt, S, skip)
    _, dev, B, _, H, G, dk, dv, ldq, ldk, ldv = _scan_sizes(q, k, v, log_alpha, dt, skip, None, 1)
    _check_f32("S", S, (B, H, dk, dv), dev)
    o = _empty_as(v)
    _raise(load().gdn2_ssm_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_alpha.data_ptr(), dt.data_ptr(), _at(skip),
                                S.data_ptr(), o.data_ptr(), ldq, ldk, ldv, B, H, G, dk, dv, _dtype_code(q),
                                _raw_stream(q)), "gdn2_ssm_step")
    return o


def _prologue_sizes(x, W, bias, xdt, dt_bias, A_log, window, cu_seqlens, lead_dims):
    if cu_seqlens is not None:
        lead_dims = 1
    xs, dtype, dev = x.shape, x.dtype, x.get_device()
    if len(xs) != lead_dims + 1 or W.dim() != 2:
        raise ValueError("x must be %s and W [C, K]" % ("[rows, C]" if lead_dims == 1 else "[B, T, C]"))
    lead, C, K = xs[:lead_dims], xs[-1], W.shape[1]
    _check_f32("W", W, (C, K), dev)
    if bias is not None:
        _check_f32("bias", bias, (C,), dev)
    H, ldt = 0, 0
    if xdt is not None:
        H = xdt.shape[-1]
        if xdt.dtype != dtype or xdt.get_device() != dev or xdt.shape[:-1] != lead or A_log is None:
            raise ValueError("xdt must be a %s tensor %s + (H,) on %s, with A_log" % (dtype, tuple(lead), x.device))
        ldt = _row_ld("xdt", xdt, lead_dims, H)
        if dt_bias is not None:
            _check_f32("dt_bias", dt_bias, (H,), dev)
        _check_f32("A_log", A_log, (H,), dev)
    if cu_seqlens is None:
        B, T = (xs[0], 1) if lead_dims == 1 else lead
    else:
        B, T = _check_cu(cu_seqlens, xs[0]), xs[0]
        if cu_seqlens.get_device() != dev:
            raise ValueError("cu_seqlens must be on %s" % x.device)
    if window is not None:
        _check_like("the window", window, (B, K - 1, C), dtype, dev)
    return dev, B, T, C, K, H, _row_ld("x", x, lead_dims, C), ldt


def ssm_prologue(x, W, bias, xdt, dt_bias, A_log, init=None, output_window=False, cu_seqlens=None, stream=None):
    """(y, dt, log_alpha, window): y = silu(conv(x) + bias) [B, T, C] with
    filters W fp32 [C, K], dt = softplus(xdt + dt_bias) and log_alpha =
    -exp(A_log) dt [B, T, H] (xdt None: neither).  init [B, K-1, C]: the inputs
    before each sequence (None: zeros); window: those before its next token
    (None without output_window).  x and xdt may be slices of wider rows.
    Packed: [rows, ..] and cu_seqlens."""
    if _elsewhere(x) or stream is not None:
        return _there(ssm_prologue, x, stream, x, W, bias, xdt, dt_bias, A_log, init, output_window, cu_seqlens)
    _, B, T, C, K, H, ldx, ldt = _prologue_sizes(x, W, bias, xdt, dt_bias, A_log, init, cu_seqlens, 2)
    y = _empty_as(x)
    dt, la = (_empty_as(xdt), _empty_as(xdt)) if H else (None, None)
    window = None
    if output_window:
        window = x.new_empty((B, K - 1, C)) if init is None else _empty_as(init)
    _raise(load().gdn2_ssm_prologue_fwd(x.data_ptr(), W.data_ptr(), _at(bias), K, _at(xdt), _at(dt_bias), _at(A_log),
                                        _at(init), y.data_ptr(), _at(dt), _at(la), _at(window), _at(cu_seqlens), ldx, ldt,
                                        B, T, C, H, _dtype_code(x), _raw_stream(x)), "gdn2_ssm_prologue_fwd")
    return y, dt, la, window


def ssm_prologue_bwd(x, W, bias, xdt, dt_bias, A_log, dy, ddt=None, dlog_alpha=None, init=None, cu_seqlens=None,
                     stream=None):
    """Gradients of ssm_prologue from dy, ddt and dlog_alpha: dx, dW, dbias,
    dxdt, ddt_bias, dA_log and, with init, dinit (None for what was not given)."""
    if _elsewhere(x) or stream is not None:
        return _there(ssm_prologue_bwd, x, stream, x, W, bias, xdt, dt_bias, A_log, dy, ddt, dlog_alpha, init, cu_seqlens)
    import torch
    dev, B, T, C, K, H, ldx, ldt = _prologue_sizes(x, W, bias, xdt, dt_bias, A_log, init, cu_seqlens, 2)
    for name, t, like in (("dy", dy, x), ("ddt", ddt, xdt), ("dlog_alpha", dlog_alpha, xdt)):
        if like is not None:
            if t is None:
                raise ValueError("%s is missing" % name)
            _check_like(name, t, like.shape, x.dtype, dev)
    e = torch.empty_like
    g = {"dx": _empty_as(x), "dW": e(W), "dbias": None if bias is None else e(bias),
         "dinit": None if init is None else e(init), "ddt_bias": e(dt_bias) if H and dt_bias is not None else None,
         "dA_log": e(A_log) if H else None, "dxdt": _empty_as(xdt) if H else None}
    nws = load().gdn2_ssm_prologue_bwd_workspace(B, T, C, K, H, cu_seqlens is not None)
    ws = _scratch(nws, x)
    _raise(load().gdn2_ssm_prologue_bwd(x.data_ptr(), W.data_ptr(), _at(bias), K, _at(xdt), _at(dt_bias), _at(A_log),
                                        _at(init), dy.data_ptr(), _at(ddt), _at(dlog_alpha), g["dx"].data_ptr(),
                                        g["dW"].data_ptr(), _at(g["dbias"]), _at(g["dxdt"]), _at(g["ddt_bias"]),
                                        _at(g["dA_log"]), _at(g["dinit"]), _at(cu_seqlens), ldx, ldt, B, T, C, H,
                                        _dtype_code(x), _at(ws), nws, _raw_stream(x)), "gdn2_ssm_prologue_bwd")
    return g


def ssm_prologue_step(x, W, bias, xdt, dt_bias, A_log, window, stream=None):
    """(y, dt, log_alpha) of one token per sequence: x [B, C], xdt [B, H]
    (None: only y); window [B, K-1, C] updated in place."""
    if _elsewhere(x) or stream is not None:
        return _there(ssm_prologue_step, x, stream, x, W, bias, xdt, dt_bias, A_log, window)
    _, B, _, C, K, H, ldx, ldt = _prologue_sizes(x, W, bias, xdt, dt_bias, A_log, window, None, 1)
    y = _empty_as(x)
    dt, la = (_empty_as(xdt), _empty_as(xdt)) if H else (None, None)
    _raise(load().gdn2_ssm_prologue_step(x.data_ptr(), W.data_ptr(), _at(bias), K, _at(xdt), _at(dt_bias), _at(A_log),
                                         _at(window), y.data_ptr(), _at(dt), _at(la), ldx, ldt, B, C, H, _dtype_code(x),
                                         _raw_stream(x)), "gdn2_ssm_prologue_step")
    return y, dt, la
