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
"""

import torch

from . import model_ops as mo
from . import poetx as px

_DTYPE = {torch.float32: px.POETX_F32, torch.bfloat16: px.POETX_BF16}
_NAME = {torch.float32: "f32", torch.bfloat16: "bf16"}


def _rows(name, t, shape, dtype, device):
    """Checks a two-dimensional tensor with contiguous rows; its row stride."""
    if t.shape != shape or t.dtype != dtype or t.device != device:
        raise ValueError(f"{name}: {tuple(t.shape)} {t.dtype} on {t.device}, expected {tuple(shape)} {dtype} on "
                         f"{device}")
    s0, s1 = t.stride()
    if s1 != 1 and shape[1] > 1:
        raise ValueError(f"{name}: the elements of a row are not contiguous (strides {s0}, {s1})")
    return s0 if shape[0] > 1 else shape[1]


def _flat(name, t, shape, dtype, device):
    """Checks a contiguous tensor."""
    if t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: {tuple(t.shape)} {t.dtype} on {t.device}, strides {t.stride()}, expected contiguous "
                         f"{tuple(shape)} {dtype} on {device}")


def _first(name, t):
    """Checks the tensor that sets an operator's shape, type and device."""
    if t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"{name}: a two-dimensional device tensor is needed, got {tuple(t.shape)} on {t.device}")
    d = _DTYPE.get(t.dtype)
    if d is None:
        raise ValueError(f"{name}: {t.dtype}, expected float32 or bfloat16")
    return t.shape, t.device, d


def _grad(t):
    """A gradient with rows of its own (autograd hands out broadcast ones)."""
    return t.contiguous() if 0 in t.stride() or t.stride(-1) != 1 else t


def _stream(device):
    """torch's current stream of the device, as a handle. Calls on another
    device than the current one run under its guard."""
    return torch.cuda.current_stream(device).cuda_stream


def rms_norm(x, gain, residual=None, eps=1e-6):
    """(h, y, rstd): h = x + residual in x's type (x itself without one), y =
    h / sqrt(mean(h^2) + eps) * gain, computed before h is rounded, and the
    rows' 1 / sqrt(...) for the backward."""
    (T, n), dev, dt = _first("x", x)
    ldx = _rows("x", x, x.shape, x.dtype, dev)
    ldr = _rows("residual", residual, x.shape, x.dtype, dev) if residual is not None else 0
    _flat("gain", gain, (n,), torch.float32, dev)
    with torch.cuda.device(dev):
        h = torch.empty((T, n), dtype=x.dtype, device=dev) if residual is not None else None
        y = torch.empty((T, n), dtype=x.dtype, device=dev)
        rstd = torch.empty(T, dtype=torch.float32, device=dev)
        mo.poetx_rmsnorm_forward(T, n, dt, x, ldx, residual, ldr, gain, eps, h, y, rstd, _stream(dev))
    return (h if h is not None else x), y, rstd


def rms_norm_q8(x, gain, residual=None, eps=1e-6):
    """(h, q, scale): the norm's rows as int8 codes with one scale a token,
    the input of ``linear_i8``."""
    (T, n), dev, dt = _first("x", x)
    ldx = _rows("x", x, x.shape, x.dtype, dev)
    ldr = _rows("residual", residual, x.shape, x.dtype, dev) if residual is not None else 0
    _flat("gain", gain, (n,), torch.float32, dev)
    with torch.cuda.device(dev):
        h = torch.empty((T, n), dtype=x.dtype, device=dev) if residual is not None else None
        q = torch.empty((T, n), dtype=torch.int8, device=dev)
        scale = torch.empty(T, dtype=torch.float32, device=dev)
        mo.poetx_rmsnorm_forward_q8(T, n, dt, x, ldx, residual, ldr, gain, eps, h, q, scale, _stream(dev))
    return (h if h is not None else x), q, scale


def quantize_rows(x):
    """(q, scale): int8 codes of x's rows with one scale a token."""
    (T, n), dev, dt = _first("x", x)
    ldx = _rows("x", x, x.shape, x.dtype, dev)
    with torch.cuda.device(dev):
        q = torch.empty((T, n), dtype=torch.int8, device=dev)
        scale = torch.empty(T, dtype=torch.float32, device=dev)
        mo.poetx_quantize_rows(T, n, dt, x, ldx, q, scale, _stream(dev))
    return q, scale


def rms_norm_backward(dy, h, rstd, gain, dh=None):
    """(dx, dgain) from dy = dL/dy and, along the residual stream, dh = dL/dh
    past the norm; dx is the gradient of x and of the residual alike."""
    dy = _grad(dy)
    (T, n), dev, dt = _first("dy", dy)
    lddy = _rows("dy", dy, dy.shape, dy.dtype, dev)
    _flat("h", h, dy.shape, dy.dtype, dev)
    _flat("rstd", rstd, (T,), torch.float32, dev)
    _flat("gain", gain, (n,), torch.float32, dev)
    lddh = 0
    if dh is not None:
        dh = _grad(dh)
        lddh = _rows("dh", dh, dy.shape, dy.dtype, dev)
    with torch.cuda.device(dev):
        dx = torch.empty((T, n), dtype=dy.dtype, device=dev)
        dgain = torch.empty(n, dtype=torch.float32, device=dev)
        ws = torch.empty(mo.poetx_rmsnorm_ws_bytes(T, n), dtype=torch.uint8, device=dev)
        mo.poetx_rmsnorm_backward(T, n, dt, dy, lddy, h, rstd, gain, dh, lddh, dx, dgain, ws, None, _stream(dev))
    return dx, dgain


def linear_i8_weight(w0):
    """wt [n][m] for ``linear_i8`` from int8 codes W0 [m][n], as
    ``DeviceLayer.export_w0`` returns them."""
    if w0.dim() != 2 or not w0.is_cuda:
        raise ValueError(f"w0: a two-dimensional device tensor is needed, got {tuple(w0.shape)} on {w0.device}")
    _flat("w0", w0, w0.shape, torch.int8, w0.device)
    m, n = w0.shape
    with torch.cuda.device(w0.device):
        wt = torch.empty((n, m), dtype=torch.int8, device=w0.device)
        mo.poetx_linear_i8_prepare(m, n, w0, wt, _stream(w0.device))
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
    with torch.cuda.device(dev):
        if out is None:
            out, ldz = torch.empty((T, n), dtype=out_dtype, device=dev), n
        else:
            ldz = _rows("out", out, (T, n), out.dtype, dev)
        dt = _DTYPE.get(out.dtype)
        if dt is None:
            raise ValueError(f"out: {out.dtype}, expected float32 or bfloat16")
        need = mo.poetx_linear_i8_ws_bytes(T, m, n)
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        mo.poetx_linear_i8(T, m, n, dt, xq, x_scale, wt, w_scale, out, ldz, ws, None, _stream(dev))
    return out


def _vocab(h, w, target, piece):
    (T, d), dev, _ = _first("h", h)
    if w.dim() != 2:
        raise ValueError(f"w: a two-dimensional tensor is needed, got {tuple(w.shape)}")
    V = w.shape[0]
    ldh = _rows("h", h, (T, d), h.dtype, dev)
    ldw = _rows("w", w, (V, d), h.dtype, dev)
    _flat("target", target, (T,), torch.int64, dev)
    return T, d, V, ldh, ldw, dev, mo.make_vocab(d, V, _NAME[h.dtype], piece)


def vocab_loss(h, w, target, piece=0):
    """(loss, lse) [T] of the softmax cross entropy of logits h w^T against
    target (int64; a target outside [0, V) is not counted: loss 0). The
    logits are not kept."""
    T, d, V, ldh, ldw, dev, D = _vocab(h, w, target, piece)
    with torch.cuda.device(dev):
        loss = torch.empty(T, dtype=torch.float32, device=dev)
        lse = torch.empty(T, dtype=torch.float32, device=dev)
        ws = torch.empty(mo.poetx_vocab_ws_bytes(D, T, mo.POETX_OP_VOCAB_FORWARD), dtype=torch.uint8, device=dev)
        mo.poetx_vocab_loss_forward(D, T, h, ldh, w, ldw, target, loss, lse, ws, None, _stream(dev))
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
    with torch.cuda.device(dev):
        dh = torch.empty((T, d), dtype=h.dtype, device=dev)
        dw = torch.empty((V, d), dtype=h.dtype, device=dev)
        ws = torch.empty(mo.poetx_vocab_ws_bytes(D, T, mo.POETX_OP_VOCAB_BACKWARD), dtype=torch.uint8, device=dev)
        mo.poetx_vocab_loss_backward(D, T, h, ldh, w, ldw, target, lse, dloss, scale, dh, dw, ws, None, _stream(dev))
    return dh, dw
