"""ctypes binding of the operators around the layer (declared in
include/poetx_model.h, exported by the same libpoetx.so).

Argument marshalling only, in the manner of ``poetx``: every function has the
name and argument order of its C counterpart, pointers may be given as ints or
as torch tensors, ``stream=None`` means torch's current HIP stream, and a
non-zero status raises ``poetx.PoetxError``. ``model`` calls these on tensors.
"""

import ctypes

from . import poetx as px
from .poetx import _I64, _P, _SZ, _call, _lib, _ptr, _size, _stream

POETX_OP_VOCAB_FORWARD, POETX_OP_VOCAB_BACKWARD = 0, 1

EXPORTED = [
    "poetx_linear_i8", "poetx_linear_i8_prepare", "poetx_quantize_rows",
    "poetx_rmsnorm_backward", "poetx_rmsnorm_forward", "poetx_rmsnorm_forward_q8", "poetx_rmsnorm_ws_bytes",
    "poetx_vocab_loss_backward", "poetx_vocab_loss_forward", "poetx_vocab_ws_bytes",
]


class poetx_vocab(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int64), ("V", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("piece", ctypes.c_int32)]


def make_vocab(d, V, dtype="bf16", piece=0):
    """poetx_vocab from sizes and a dtype name ("f32", "bf16")."""
    return poetx_vocab(d, V, px._DTYPES[dtype], piece)


_D = ctypes.POINTER(poetx_vocab)
_INT, _F = ctypes.c_int, ctypes.c_float
_sig = {
    "poetx_rmsnorm_forward": (_INT, [_I64, _I64, _INT, _P, _I64, _P, _I64, _P, _F, _P, _P, _P, _P]),
    "poetx_rmsnorm_forward_q8": (_INT, [_I64, _I64, _INT, _P, _I64, _P, _I64, _P, _F, _P, _P, _P, _P]),
    "poetx_quantize_rows": (_INT, [_I64, _I64, _INT, _P, _I64, _P, _P, _P]),
    "poetx_rmsnorm_backward": (_INT, [_I64, _I64, _INT, _P, _I64, _P, _P, _P, _P, _I64, _P, _P, _P, _SZ, _P]),
    "poetx_rmsnorm_ws_bytes": (_SZ, [_I64, _I64]),
    "poetx_linear_i8": (_INT, [_I64, _I64, _I64, _INT, _P, _P, _P, _P, _P, _I64, _P]),
    "poetx_linear_i8_prepare": (_INT, [_I64, _I64, _P, _P, _P]),
    "poetx_vocab_ws_bytes": (_SZ, [_D, _I64, _INT]),
    "poetx_vocab_loss_forward": (_INT, [_D, _I64, _P, _I64, _P, _I64, _P, _P, _P, _P, _SZ, _P]),
    "poetx_vocab_loss_backward": (_INT, [_D, _I64, _P, _I64, _P, _I64, _P, _P, _P, _F, _P, _P, _P, _SZ, _P]),
}
for _name, (_res, _args) in _sig.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args


def poetx_rmsnorm_forward(T, n, dtype, x, ldx, res, ldr, gain, eps, h, y, rstd, stream=None):
    _call("poetx_rmsnorm_forward", T, n, dtype, _ptr(x), ldx, _ptr(res), ldr, _ptr(gain), eps, _ptr(h), _ptr(y),
          _ptr(rstd), _stream(stream))


def poetx_rmsnorm_forward_q8(T, n, dtype, x, ldx, res, ldr, gain, eps, h, q, q_scale, stream=None):
    _call("poetx_rmsnorm_forward_q8", T, n, dtype, _ptr(x), ldx, _ptr(res), ldr, _ptr(gain), eps, _ptr(h), _ptr(q),
          _ptr(q_scale), _stream(stream))


def poetx_quantize_rows(T, n, dtype, x, ldx, q, q_scale, stream=None):
    _call("poetx_quantize_rows", T, n, dtype, _ptr(x), ldx, _ptr(q), _ptr(q_scale), _stream(stream))


def poetx_rmsnorm_backward(T, n, dtype, dy, lddy, h, rstd, gain, dh, lddh, dx, dgain, ws=None, ws_bytes=None,
                           stream=None):
    _call("poetx_rmsnorm_backward", T, n, dtype, _ptr(dy), lddy, _ptr(h), _ptr(rstd), _ptr(gain), _ptr(dh), lddh,
          _ptr(dx), _ptr(dgain), _ptr(ws), _size(ws, ws_bytes), _stream(stream))


def poetx_rmsnorm_ws_bytes(T, n):
    return _lib.poetx_rmsnorm_ws_bytes(T, n)


def poetx_linear_i8(T, m, n, out_dtype, xq, x_scale, wt, w_scale, z, ldz, stream=None):
    _call("poetx_linear_i8", T, m, n, out_dtype, _ptr(xq), _ptr(x_scale), _ptr(wt), _ptr(w_scale), _ptr(z), ldz,
          _stream(stream))


def poetx_linear_i8_prepare(m, n, w0, wt, stream=None):
    _call("poetx_linear_i8_prepare", m, n, _ptr(w0), _ptr(wt), _stream(stream))


def poetx_vocab_ws_bytes(D, T, op):
    return _lib.poetx_vocab_ws_bytes(ctypes.byref(D), T, op)


def poetx_vocab_loss_forward(D, T, h, ldh, w, ldw, target, loss, lse, ws=None, ws_bytes=None, stream=None):
    _call("poetx_vocab_loss_forward", ctypes.byref(D), T, _ptr(h), ldh, _ptr(w), ldw, _ptr(target), _ptr(loss),
          _ptr(lse), _ptr(ws), _size(ws, ws_bytes), _stream(stream))


def poetx_vocab_loss_backward(D, T, h, ldh, w, ldw, target, lse, dloss, scale, dh, dw, ws=None, ws_bytes=None,
                              stream=None):
    _call("poetx_vocab_loss_backward", ctypes.byref(D), T, _ptr(h), ldh, _ptr(w), ldw, _ptr(target), _ptr(lse),
          _ptr(dloss), scale, _ptr(dh), _ptr(dw), _ptr(ws), _size(ws, ws_bytes), _stream(stream))
