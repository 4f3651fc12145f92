"""Log probabilities and their gradients in workspaces of the queried size and of the least
that is taken, for which the vocabulary's pieces shrink and products are not split, with known
bytes behind the workspace's end; and sizes of one operator that are reached by few calls:
hidden rows past what a workgroup keeps, and alternatives without targets some tokens at a time."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from model_cases import U16, U32, f64, normal, within  # noqa: E402
from oracle import model_oracle as M  # noqa: E402
from orthogonal_equivalence_amd import model  # noqa: E402
from orthogonal_equivalence_amd import model_ops as mo  # noqa: E402
from orthogonal_equivalence_amd import poetx as px  # noqa: E402
from test_gpu_token_logprobs import _check, _inputs  # noqa: E402

GUARD = 1 << 16
TAU = 0.9


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible AMD GPU"
    torch.cuda.init()


class Guarded:
    """A workspace whose bytes are 0xff (NaN wherever one is read unwritten) in a buffer of
    0xa5 bytes."""

    def __init__(self, size):
        self.all = torch.full((GUARD + size + GUARD,), 0xa5, dtype=torch.uint8, device="cuda")
        self.ws, self.size = self.all[GUARD:GUARD + size], size
        self.ws.fill_(0xff)

    def check(self):
        assert torch.all(self.all[:GUARD] == 0xa5) and torch.all(self.all[GUARD + self.size:] == 0xa5)


def _least(call, high):
    """The least size with which call(null workspace, size) is not refused for it."""
    def taken(size):
        with pytest.raises(px.PoetxError) as e:
            call(None, size)
        return e.value.status == px.POETX_EINVAL

    low = 0
    while high - low > 1:
        mid = (low + high) // 2
        low, high = (low, mid) if taken(mid) else (mid, high)
    return high


def _forward(D, h, w, t, top):
    T = h.shape[0]
    out = [torch.full((T,) + s, 7.0, device="cuda") for s in ((), (), (2,))]
    ids = torch.full((T, top), 9, device="cuda") if top else None
    alt = torch.full((T, top), 7.0, device="cuda") if top else None

    def call(ws, size):
        mo.poetx_token_logprobs(D, T, TAU, h, h.shape[1], w, w.shape[1], t, top, out[0], out[1], out[2], ids, alt, ws, size)

    return out + [ids, alt], call


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("top", [0, 5, 64])
@pytest.mark.parametrize("T,d,V", [(5, 72, 3001), (130, 64, 20000), (700, 136, 2500), (9001, 64, 300)])
def test_forward(T, d, V, top, act):
    print(f"\n[gpu] guarded forward T={T} d={d} V={V} top={top} {act}", flush=True)
    rng = np.random.default_rng([T, V])
    h, w, t = _inputs(rng, T, d, V, act)
    D = mo.make_vocab(d, V, act)
    want = model.token_logprobs(h, w, t, top=top, temperature=TAU)
    full = mo.poetx_token_ws_bytes(D, T, mo.POETX_OP_VOCAB_FORWARD, top)
    out, call = _forward(D, h, w, t, top)
    for size in (full, _least(call, full)):
        ws = Guarded(size)
        call(ws.ws, size)
        torch.cuda.synchronize()
        ws.check()
        # sums of up to 136 products in another order: 4 (d / 2 + 2 + 100) u32 of sum |h w|, under 150
        for a, b in zip(want[:3], out[:3]):
            assert torch.allclose(a, b, rtol=1e-4, atol=4 * (d / 2 + 102) * U32 * 150)
        if top:
            assert torch.equal(want[3], out[3])


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,V", [(3, 72, 5000), (70, 264, 20000), (700, 136, 2500), (2500, 512, 3000), (9001, 64, 300)])
def test_backward(T, d, V, act):
    print(f"\n[gpu] guarded backward T={T} d={d} V={V} {act}", flush=True)
    rng = np.random.default_rng([T, V])
    h, w, t = _inputs(rng, T, d, V, act)
    a, b = normal(rng, T, "f32"), normal(rng, T, "f32", 0.3)
    D = mo.make_vocab(d, V, act)
    _, entropy, stat, _, _ = model.token_logprobs(h, w, t, temperature=TAU)
    H, W, N = f64(h), f64(w), t.cpu().numpy()
    _, ENT, LSE, ALL, counted = M.token_logprobs(H, W, N, TAU)
    P = np.where(counted[:, None], np.exp(ALL), 0.0)
    sums = (np.abs(H) @ np.abs(W).T).max(1)
    off = (d / 16 + 16 if act == "bf16" else d / 2 + 2) * U32 * sums / TAU + 100 * U32 * (np.abs(LSE) + 10)
    r16 = U16 if act == "bf16" else 0.0
    chain = (max(T, V) / 16 + 16 if act == "bf16" else max(T, V) / 2 + 2) * U32
    full = mo.poetx_token_ws_bytes(D, T, mo.POETX_OP_VOCAB_BACKWARD)
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    for da, db in ((a, b), (a, None), (None, b)):
        A, B = (np.zeros((T, 1)) if x is None else f64(x)[:, None] for x in (da, db))
        DH, DW, _ = M.token_logprobs_backward(H, W, N, A[:, 0], B[:, 0], TAU)
        size = np.abs(A) * P + np.abs(B) * P * np.abs(ALL + ENT[:, None])
        size[counted, N[counted]] += 2 * np.abs(A)[counted, 0]
        err = ((3 * off[:, None] + r16 + 16 * U32 + chain) * size + 4 * off[:, None] * np.abs(B) * P * (2 + ENT[:, None])) / TAU

        def call(ws, size):
            mo.poetx_token_logprobs_backward(D, T, TAU, h, d, w, d, t, stat, entropy, da, db, dh, dw, ws, size)

        least = _least(call, full)
        print(f"[gpu] {full} bytes, least {least}", flush=True)
        for n in (full, (full + least) // 2, least):
            ws = Guarded(n)
            dh.fill_(5.0)
            dw.fill_(5.0)
            call(ws.ws, n)
            torch.cuda.synchronize()
            ws.check()
            within("dh", dh, DH, r16 * np.abs(DH) + err @ np.abs(W) + 1e-30)
            within("dw", dw, DW, r16 * np.abs(DW) + err.T @ np.abs(np.where(counted[:, None], H, 0.0)) + 1e-30)


@pytest.mark.parametrize("act,d", [("bf16", 8200), ("bf16", 20480), ("f32", 4104), ("f32", 8192)])
@pytest.mark.parametrize("T,V,top", [(1, 3000, 5), (300, 500, 20), (520, 300, 64)])
def test_long_hidden_rows_with_alternatives(T, V, top, act, d):
    """Past 16 KB a row."""
    print(f"\n[gpu] token_logprobs T={T} d={d} V={V} top={top} {act}", flush=True)
    rng = np.random.default_rng([T, d])
    h, w, t = _inputs(rng, T, d, V, act)
    _check(h, w, t, act, top, grads=False)
    _check(h, w, None, act, top, grads=False)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(600, 1100000), (2001, 270000)])
def test_alternatives_without_targets_some_tokens_at_a_time(T, V, act):
    """1 GB of logits: 256 tokens of 1100000, 1792 of 270000. Rows one after the other, and far
    apart, which come gathered."""
    d, top = 64, 20
    print(f"\n[gpu] token_logprobs T={T} d={d} V={V} top={top} {act}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(T)
    dt = torch.bfloat16 if act == "bf16" else torch.float32
    h = torch.randn((T, d), generator=g, device="cuda").to(dt)
    w = (0.25 * torch.randn((V, d), generator=g, device="cuda")).to(dt)
    _, entropy, stat, ids, alt = model.token_logprobs(h, w, top=top)
    wd = w.double()
    for i in range(0, T, 200):
        print(f"[gpu] rows from {i}", flush=True)
        lp = torch.log_softmax(h[i:i + 200].double() @ wd.t(), 1)
        value, at = torch.sort(lp, dim=1, descending=True, stable=True)
        assert torch.equal(ids[i:i + 200], at[:, :top])
        # logits of up to 15 in sums of 64 products (66 u32 sum |h w| < 1e-4) and their lse
        within("alternatives", alt[i:i + 200], f64(value[:, :top]), 4e-4)
        within("entropy", entropy[i:i + 200], f64(-(lp.exp() * lp).sum(1)), 4e-3)
    far = torch.empty((T - 1) * ((1 << 22) + 64) + d, dtype=dt, device="cuda").as_strided((T, d), ((1 << 22) + 64, 1))
    far.copy_(h)
    for a, b in zip((entropy, stat, ids, alt), model.token_logprobs(far, w, top=top)[1:]):
        assert torch.equal(a, b)
