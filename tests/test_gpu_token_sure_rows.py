"""Gradients of rows that are sure of a token, where the backward's logits come from tiles
that sum in another order than the forward's: other vocabulary pieces, other workspaces,
alternatives held some tokens at a time.

A logit is off by `off` whatever the order, and so every exponential by twice that share of
itself, what is composed of the others' by as much; the largest logit's own distance is 0 and
1 - p is formed from the others' sum. Nothing of the size of a logit's rounding, 1e-5 of the
upstream gradient at logits of 300, may be left where the terms are 1e-10 of it."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from model_cases import DTYPES, U16, U32, f64, normal, within  # noqa: E402
from orthogonal_equivalence_amd import model  # noqa: E402
from orthogonal_equivalence_amd import model_ops as mo  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible AMD GPU"
    torch.cuda.init()


def _backward(h, w, t, stat, entropy, a, b, tau, piece, ws_bytes=None):
    (T, d), V = h.shape, w.shape[0]
    D = mo.make_vocab(d, V, "bf16" if h.dtype == torch.bfloat16 else "f32", piece)
    need = mo.poetx_token_ws_bytes(D, T, mo.POETX_OP_VOCAB_BACKWARD) if ws_bytes is None else ws_bytes
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
    dh, dw = torch.full_like(h, 3.0), torch.full_like(w, 3.0)
    mo.poetx_token_logprobs_backward(D, T, tau, h, d, w, d, t, stat, entropy, a, b, dh, dw, ws)
    return dh, dw


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("second", [False, True])
@pytest.mark.parametrize("tau", [1.0, 0.25])
@pytest.mark.parametrize("T,V,piece", [(64, 900, 0), (64, 900, 256), (64, 20000, 256), (64, 20000, 4096), (300, 9000, 256),
                                       (300, 9000, 0), (700, 5000, 512)])
def test_pieces(T, V, piece, tau, second, act):
    """`second`: half of the targets are not the token that the row is sure of."""
    print(f"\n[gpu] sure rows T={T} V={V} piece={piece} tau={tau} {act}", flush=True)
    rng = np.random.default_rng([T, V])
    d = 264
    w = rng.standard_normal((V, d))
    w /= np.linalg.norm(w, axis=1, keepdims=True)
    sure = rng.integers(0, V, T)
    h = torch.from_numpy((w[sure] * np.linspace(20, 300, T)[:, None] * tau).astype(np.float32)).to(DTYPES[act]).cuda()
    w = torch.from_numpy(w.astype(np.float32)).to(DTYPES[act]).cuda()
    t = np.where(rng.random(T) < 0.5, (sure + 1) % V, sure) if second else sure
    tt = torch.from_numpy(t).cuda()
    _, entropy, stat, _, _ = model.token_logprobs(h, w, tt, temperature=tau)
    L = f64(h) @ f64(w).T / tau
    X = L - L.max(1, keepdims=True)
    most = L.argmax(1)
    assert (most == sure).all()
    each = np.arange(T)
    E = np.exp(X)
    E[each, most] = 0.0
    rest = E.sum(1)
    P = np.exp(X) / (1 + rest)[:, None]
    LOGP = X - np.log1p(rest)[:, None]
    ENT = np.log1p(rest) - (P * X).sum(1)
    off = (d / 16 + 16 if act == "bf16" else d / 2 + 2) * U32 * (np.abs(f64(h)) @ np.abs(f64(w)).T).max(1) / tau
    rel = 4 * off + (80 + 6 * np.abs(X).max(1)) * U32
    tiny = V * 2.0 ** -126
    r16 = U16 if act == "bf16" else 4 * U32
    chain = ((max(T, V) / 16 + 16) if act == "bf16" else (max(T, V) / 2 + 2)) * U32
    a, b = normal(rng, T, "f32"), normal(rng, T, "f32")
    for da, db in ((a, None), (None, b), (a, b)):
        A, B = (np.zeros((T, 1)) if x is None else f64(x)[:, None] for x in (da, db))
        DL = -A * P - B * P * (LOGP + ENT[:, None])
        size = np.abs(A) * P + np.abs(B) * P * (np.abs(LOGP) + ENT[:, None])
        if da is not None:
            # 1 - p of the target, not by that difference where p is near 1
            miss, PT = np.where(t == most, rest / (1 + rest), 1.0 - P[each, t]), P[each, t]
            DL[each, t] = A[:, 0] * miss - B[:, 0] * PT * (LOGP[each, t] + ENT)
            size[each, t] = np.abs(A[:, 0]) * miss + np.abs(B[:, 0]) * PT * (np.abs(LOGP[each, t]) + ENT)
        DH, DW = DL @ f64(w) / tau, DL.T @ f64(h) / tau
        dh, dw = _backward(h, w, tt, stat, entropy, da, db, tau, piece)
        torch.cuda.synchronize()
        # what a bfloat16 or float term below the smallest normal number loses, of the unit
        err = ((2 * rel[:, None] + r16 + chain) * size + 90 * tiny * (np.abs(A).max() + np.abs(B).max())) / tau
        within("dh", dh, DH, r16 * np.abs(DH) + 1.01 * err @ np.abs(f64(w)) + 1e-37)
        within("dw", dw, DW, r16 * np.abs(DW) + 1.01 * err.T @ np.abs(f64(h)) + 1e-37)
