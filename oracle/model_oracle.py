"""float64 NumPy forms of the operators around the layer, written from their
formulas: the RMS norm of the residual stream and its gradients, int8 rows
with one scale each, the int8 product, and the softmax cross entropy over a
vocabulary with its gradients. No code of the library is used."""

import numpy as np


def rms_norm(x, gain, residual=None, eps=1e-6):
    """(h, y, rstd) with h = x + residual, y = h / sqrt(mean(h^2) + eps) * gain."""
    h = np.asarray(x, np.float64) + (0.0 if residual is None else np.asarray(residual, np.float64))
    rstd = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
    return h, h * rstd[:, None] * np.asarray(gain, np.float64), rstd


def rms_norm_backward(dy, h, gain, eps=1e-6, dh=None, rstd=None):
    """(dx, dgain) of sum(dy * y) + sum(dh * h); rstd: the forward's, where h
    was rounded after it was taken."""
    dy, h, gain = (np.asarray(a, np.float64) for a in (dy, h, gain))
    if rstd is None:
        rstd = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
    u = h * np.asarray(rstd, np.float64)[:, None]
    dyg = dy * gain
    dx = np.asarray(rstd, np.float64)[:, None] * (dyg - u * np.mean(dyg * u, axis=1, keepdims=True))
    if dh is not None:
        dx = dx + np.asarray(dh, np.float64)
    return dx, np.sum(dy * u, axis=0)


def quantize_rows(y):
    """(codes, scale): scale = max|y| / 127 per row (1 for a row below
    2^-100, whose codes are 0), codes = rint(y / scale)."""
    y = np.asarray(y, np.float64)
    a = np.max(np.abs(y), axis=1)
    zero = a < 2.0 ** -100
    scale = np.where(zero, 1.0, a / 127.0)
    return np.where(zero[:, None], 0.0, np.rint(y / scale[:, None])), scale


def linear_i8(xq, x_scale, wt, w_scale):
    """z[t][c] = x_scale[t] w_scale[c] sum_k xq[t][k] wt[c][k] (the sums are
    whole numbers below 2^53, exact in float64)."""
    s = np.asarray(xq, np.float64) @ np.asarray(wt, np.float64).T
    return s * np.asarray(x_scale, np.float64)[:, None] * np.asarray(w_scale, np.float64)[None, :]


def vocab_loss(h, w, target):
    """(loss, lse, counted): softmax cross entropy of the rows h w^T; rows
    whose target is outside [0, V) have loss and lse 0 and are never read."""
    w, target = np.asarray(w, np.float64), np.asarray(target)
    V = w.shape[0]
    counted = (target >= 0) & (target < V)
    loss, lse = np.zeros(len(target)), np.zeros(len(target))
    if counted.any():
        l = np.asarray(h, np.float64)[counted] @ w.T
        top = l.max(axis=1)
        z = top + np.log(np.sum(np.exp(l - top[:, None]), axis=1))
        lse[counted] = z
        loss[counted] = z - l[np.arange(len(z)), target[counted]]
    return loss, lse, counted


def vocab_loss_backward(h, w, target, g):
    """(dh, dw, dl) of sum_t g[t] loss[t]; dl [T][V] is the gradient of the
    logits (0 in rows that are not counted)."""
    w, target, g = np.asarray(w, np.float64), np.asarray(target), np.asarray(g, np.float64)
    T, V = len(target), w.shape[0]
    _, lse, counted = vocab_loss(h, w, target)
    hc = np.asarray(h, np.float64)[counted]
    p = np.exp(hc @ w.T - lse[counted][:, None])
    p[np.arange(len(p)), target[counted]] -= 1.0
    dl = np.zeros((T, V))
    dl[counted] = p * g[counted][:, None]
    dh = dl @ w
    return dh, dl[counted].T @ hc, dl
