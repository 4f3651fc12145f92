"""The operators around a POET-X layer, on torch tensors: the RMS norm of the
residual stream, the int8 product that serves a merged quantised layer, and
the vocabulary cross entropy.

Every function checks its tensors, allocates its outputs and workspace with
torch's allocator on the current stream, and makes one call of the C ABI
(``model_ops``) on that stream; all arithmetic runs in libpoetx.so. A tensor
made on another stream has to be ordered before the call by the caller, as
for any torch operation. Two-dimensional inputs may have any row stride whose
rows start on 16-byte boundaries; gradients that come in broadcast (expanded)
are copied out first.

The functions record no graph: gradients come from the ``_backward`` functions.
While torch records gradients, an input that requires one is refused, as its
results would silently be cut off from it; call them under ``torch.no_grad()``
or within a ``torch.autograd.Function``.
"""

import torch

from . import model_ops as mo
from . import poetx as px
from .poetx import _lib

_DTYPE = {torch.float32: px.POETX_F32, torch.bfloat16: px.POETX_BF16}
_NAME = {torch.float32: "f32", torch.bfloat16: "bf16"}


def _requires_grad(name, t):
    """Refuses an input that requires a gradient, where torch records them."""
    if torch.is_grad_enabled():
        raise ValueError(f"{name}: {tuple(t.shape)} requires a gradient, and no graph is recorded here: call under "
                         "torch.no_grad() and take gradients from the _backward functions")


def _rows(name, t, shape, dtype, device):
    """Checks a two-dimensional tensor with contiguous rows; its row stride."""
    if t.shape != shape or t.dtype != dtype or t.device != device:
        raise ValueError(f"{name}: {tuple(t.shape)} {t.dtype} on {t.device}, expected {tuple(shape)} {dtype} on "
                         f"{device}")
    return _stride(name, t, shape)


def _stride(name, t, shape):
    if t.requires_grad:
        _requires_grad(name, t)
    s0, s1 = t.stride()
    if s1 != 1 and shape[1] > 1:
        raise ValueError(f"{name}: the elements of a row are not contiguous (strides {s0}, {s1})")
    return s0 if shape[0] > 1 else shape[1]


def _flat(name, t, shape, dtype, device):
    """Checks a contiguous tensor."""
    if t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: {tuple(t.shape)} {t.dtype} on {t.device}, strides {t.stride()}, expected contiguous "
                         f"{tuple(shape)} {dtype} on {device}")
    if t.requires_grad:
        _requires_grad(name, t)


def _first(name, t):
    """Checks the tensor that sets an operator's shape, type and device; those
    and its row stride."""
    d, shape = _DTYPE.get(t.dtype), t.shape
    if d is None or len(shape) != 2 or not t.is_cuda:
        raise ValueError(f"{name}: a two-dimensional float32 or bfloat16 device tensor is needed, got "
                         f"{tuple(shape)} {t.dtype} on {t.device}")
    return shape, t.device, d, _stride(name, t, shape)


def _grad(t):
    """A gradient with rows of its own (autograd hands out broadcast ones)."""
    s = t.stride()
    return t.contiguous() if s and (0 in s or s[-1] != 1) else t  # (a scalar is refused with its shape)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _call(f, dev, *args):
    """The entry point on torch's current stream of the tensors' device (its
    raw handle: a call's host time is a few microseconds, and a Stream object
    would cost two), with that device current for the launches."""
    i = dev.index
    if i != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            st = f(*args, torch._C._cuda_getCurrentRawStream(i))
    else:
        st = f(*args, torch._C._cuda_getCurrentRawStream(i))
    if st != px.POETX_OK:
        raise px.PoetxError(f.__name__, st)


def _like(t):
    """A contiguous tensor of t's shape and type."""
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


def _new(rows, cols, dtype, dev):
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=dev)


def _scratch(need, dev):
    return torch.empty(need, dtype=torch.uint8, device=dev) if need else None


def rms_norm(x, gain, residual=None, eps=1e-6):
    """(h, y, rstd): h = x + residual in x's type (x itself without one), y =
    h / sqrt(mean(h^2) + eps) * gain, computed before h is rounded, and the
    rows' 1 / sqrt(...) for the backward."""
    shape, dev, dt, ldx = _first("x", x)
    T, n = shape
    ldr = _rows("residual", residual, shape, x.dtype, dev) if residual is not None else 0
    _flat("gain", gain, (n,), torch.float32, dev)
    h = _like(x) if residual is not None else None
    y = _like(x)
    rstd = gain.new_empty(T)
    _call(_lib.poetx_rmsnorm_forward, dev, T, n, dt, x.data_ptr(), ldx, _ptr(residual), ldr, gain.data_ptr(), eps,
          _ptr(h), y.data_ptr(), rstd.data_ptr())
    return (h if h is not None else x), y, rstd


def rms_norm_q8(x, gain, residual=None, eps=1e-6):
    """(h, q, scale): the norm's rows as int8 codes with one scale a token,
    the input of ``linear_i8``."""
    shape, dev, dt, ldx = _first("x", x)
    T, n = shape
    ldr = _rows("residual", residual, shape, x.dtype, dev) if residual is not None else 0
    _flat("gain", gain, (n,), torch.float32, dev)
    h = _like(x) if residual is not None else None
    q = _new(T, n, torch.int8, dev)
    scale = gain.new_empty(T)
    _call(_lib.poetx_rmsnorm_forward_q8, dev, T, n, dt, x.data_ptr(), ldx, _ptr(residual), ldr, gain.data_ptr(), eps,
          _ptr(h), q.data_ptr(), scale.data_ptr())
    return (h if h is not None else x), q, scale


def quantize_rows(x):
    """(q, scale): int8 codes of x's rows with one scale a token."""
    (T, n), dev, dt, ldx = _first("x", x)
    q = _new(T, n, torch.int8, dev)
    scale = torch.empty(T, dtype=torch.float32, device=dev)
    _call(_lib.poetx_quantize_rows, dev, T, n, dt, x.data_ptr(), ldx, q.data_ptr(), scale.data_ptr())
    return q, scale


def rms_norm_backward(dy, h, rstd, gain, dh=None):
    """(dx, dgain) from dy = dL/dy and, along the residual stream, dh = dL/dh
    past the norm; dx is the gradient of x and of the residual alike."""
    dy = _grad(dy)
    (T, n), dev, dt, lddy = _first("dy", dy)
    h = h if h.is_contiguous() else h.contiguous()  # without a residual h is the caller's x, of any row stride
    _flat("h", h, dy.shape, dy.dtype, dev)
    _flat("rstd", rstd, (T,), torch.float32, dev)
    _flat("gain", gain, (n,), torch.float32, dev)
    lddh = 0
    if dh is not None:
        dh = _grad(dh)
        lddh = _rows("dh", dh, dy.shape, dy.dtype, dev)
    dx = _like(dy)
    dgain = torch.empty_like(gain)
    need = mo.poetx_rmsnorm_ws_bytes(T, n)
    ws = _scratch(need, dev)
    _call(_lib.poetx_rmsnorm_backward, dev, T, n, dt, dy.data_ptr(), lddy, h.data_ptr(), rstd.data_ptr(),
          gain.data_ptr(), _ptr(dh), lddh, dx.data_ptr(), dgain.data_ptr(), _ptr(ws), need)
    return dx, dgain


def linear_i8_weight(w0):
    """wt [n][m] for ``linear_i8`` from int8 codes W0 [m][n], as
    ``DeviceLayer.export_w0`` returns them."""
    if w0.dim() != 2 or not w0.is_cuda:
        raise ValueError(f"w0: a two-dimensional device tensor is needed, got {tuple(w0.shape)} on {w0.device}")
    _flat("w0", w0, w0.shape, torch.int8, w0.device)
    m, n = w0.shape
    wt = torch.empty((n, m), dtype=torch.int8, device=w0.device)
    _call(_lib.poetx_linear_i8_prepare, w0.device, m, n, w0.data_ptr(), wt.data_ptr())
    return wt


def linear_i8(xq, x_scale, wt, w_scale, out_dtype=torch.bfloat16, out=None):
    """z[t][c] = x_scale[t] w_scale[c] sum_k xq[t][k] wt[c][k]. ``out``: a
    [T][n] tensor (rows of any stride) to write to."""
    if xq.dim() != 2 or wt.dim() != 2 or not xq.is_cuda:
        raise ValueError(f"xq, wt: two-dimensional device tensors are needed, got {tuple(xq.shape)}, {tuple(wt.shape)}")
    dev = xq.device
    (T, m), n = xq.shape, wt.shape[0]
    _flat("xq", xq, (T, m), torch.int8, dev)
    _flat("x_scale", x_scale, (T,), torch.float32, dev)
    _flat("wt", wt, (n, m), torch.int8, dev)
    _flat("w_scale", w_scale, (n,), torch.float32, dev)
    if out is None:
        out, ldz = _new(T, n, out_dtype, dev), n
    else:
        ldz = _rows("out", out, (T, n), out.dtype, dev)
    dt = _DTYPE.get(out.dtype)
    if dt is None:
        raise ValueError(f"out: {out.dtype}, expected float32 or bfloat16")
    _call(_lib.poetx_linear_i8, dev, T, m, n, dt, xq.data_ptr(), x_scale.data_ptr(), wt.data_ptr(), w_scale.data_ptr(),
          out.data_ptr(), ldz)
    return out


def _vocab(h, w, target, piece):
    (T, d), dev, _, ldh = _first("h", h)
    if w.dim() != 2:
        raise ValueError(f"w: a two-dimensional tensor is needed, got {tuple(w.shape)}")
    V = w.shape[0]
    ldw = _rows("w", w, (V, d), h.dtype, dev)
    _flat("target", target, (T,), torch.int64, dev)
    return T, d, V, ldh, ldw, dev, mo.make_vocab(d, V, _NAME[h.dtype], piece)


def vocab_loss(h, w, target, piece=0):
    """(loss, lse) [T] of the softmax cross entropy of logits h w^T against
    target (int64; a target outside [0, V) is not counted: loss 0). The
    logits are not kept."""
    T, d, V, ldh, ldw, dev, D = _vocab(h, w, target, piece)
    loss = torch.empty(T, dtype=torch.float32, device=dev)
    lse = torch.empty_like(loss)
    need = mo.poetx_vocab_ws_bytes(D, T, mo.POETX_OP_VOCAB_FORWARD)
    ws = _scratch(need, dev)
    _call(_lib.poetx_vocab_loss_forward, dev, D, T, h.data_ptr(), ldh, w.data_ptr(), ldw, target.data_ptr(),
          loss.data_ptr(), lse.data_ptr(), _ptr(ws), need)
    return loss, lse


def vocab_loss_backward(h, w, target, lse, dloss=None, scale=1.0, piece=0):
    """(dh, dw) for the loss gradients scale * dloss [T] or, without dloss,
    for scale times the mean loss over the counted tokens. ``piece``:
    vocabulary rows whose gradients are held at a time (0: chosen)."""
    T, d, V, ldh, ldw, dev, D = _vocab(h, w, target, piece)
    _flat("lse", lse, (T,), torch.float32, dev)
    if dloss is not None:
        dloss = _grad(dloss)
        _flat("dloss", dloss, (T,), torch.float32, dev)
    dh, dw = _like(h), _like(w)
    need = mo.poetx_vocab_ws_bytes(D, T, mo.POETX_OP_VOCAB_BACKWARD)
    ws = _scratch(need, dev)
    _call(_lib.poetx_vocab_loss_backward, dev, D, T, h.data_ptr(), ldh, w.data_ptr(), ldw, target.data_ptr(),
          lse.data_ptr(), _ptr(dloss), scale, dh.data_ptr(), dw.data_ptr(), _ptr(ws), need)
    return dh, dw
