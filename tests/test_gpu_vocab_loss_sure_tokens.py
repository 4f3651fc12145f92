"""Softmax cross entropy of tokens that the model is sure of: the loss is a
small number beside large logits, and never negative.

Every logit here is one product of two bfloat16 values (the other features of a
row are zero) and exact in float32, so that only the softmax's own roundings
count. Bounds in units of u32, each step's rounding in its order: a tile's sum
of exponentials holds the exponential of its maximum (5 at most, none where the
difference is taken first), its logarithm 1 ulp of the result or of the argument near 1 (4). Terms
beside the maximum are off by their exponent's size, at most 36, plus the sums'
and the difference's roundings, all relative to terms that are at most the loss
itself.
"""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from model_cases import DTYPES, U32, f64, within  # noqa: E402
from oracle import model_oracle as M  # noqa: E402
from orthogonal_equivalence_amd import model  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible AMD GPU"
    torch.cuda.init()


def _bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).bfloat16().float()


def _case(T, V, d, act, size, others, seed):
    """h, w, target with logits a_t b_v: b = about 1 at the target's column and
    `others` elsewhere; feature 8 + t marks token t and meets zeros in w."""
    rng = np.random.default_rng([T, V, seed])
    h, w = torch.zeros(T, d), torch.zeros(V, d)
    h[:, 0] = _bf16(rng.uniform(size[0], size[1], T))
    w[:, 0] = _bf16(rng.uniform(others[0], others[1], V))
    y = int(rng.integers(0, V))
    w[y, 0] = _bf16(rng.uniform(1.0, 1.25))
    if d >= 8 + T:
        h[range(T), range(8, 8 + T)] = 1.0
    t = torch.full((T,), y, dtype=torch.int64)
    return h.to(DTYPES[act]).cuda(), w.to(DTYPES[act]).cuda(), t.cuda()


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("V", [2, 300, 3001, 40000])
def test_a_sure_token_has_no_loss(V, act):
    print(f"\n[gpu] vocab_loss sure tokens V={V} {act}", flush=True)
    h, w, t = _case(200, V, 64, act, (60.0, 300.0), (-1.0, 0.0), 0)
    loss, lse = model.vocab_loss(h, w, t)
    torch.cuda.synchronize()
    LOSS, LSE, _ = M.vocab_loss(f64(h), f64(w), t.cpu().numpy())
    assert LOSS.max() < 1e-20
    assert float(loss.min()) >= 0.0
    within("loss", loss, LOSS, 16 * U32)
    within("lse", lse, LSE, 16 * U32 + U32 * np.abs(LSE))


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("at", [0, 1])
def test_small_and_large_losses_beside_large_logits(at, act):
    """Two words, the target the likelier or the less likely one."""
    rng = np.random.default_rng(5)
    T = 300
    h, w = torch.zeros(T, 64), torch.zeros(2, 64)
    h[:, 0] = _bf16(rng.uniform(60.0, 250.0, T))
    w[:, 0] = torch.tensor([1.0, 0.90625])  # differences of 5.6 to 23.4
    h, w = h.to(DTYPES[act]).cuda(), w.to(DTYPES[act]).cuda()
    t = torch.full((T,), at, dtype=torch.int64, device="cuda")
    loss, _ = model.vocab_loss(h, w, t)
    torch.cuda.synchronize()
    LOSS, _, _ = M.vocab_loss(f64(h), f64(w), t.cpu().numpy())
    assert float(loss.min()) >= 0.0
    within("loss", loss, LOSS, (16 + 52 * LOSS) * U32)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_the_targets_term_of_a_sure_token_keeps_its_sign(sign, act):
    """dl = g (p - 1) at the target, read off dw through the features that mark
    the tokens: between 0 and the rounding of lse, never past 0."""
    T, V = 100, 700
    h, w, t = _case(T, V, 112, act, (60.0, 300.0), (-1.0, 0.0), 1)
    _, lse = model.vocab_loss(h, w, t)
    dloss = torch.full((T,), sign, device="cuda")
    _, dw = model.vocab_loss_backward(h, w, t, lse, dloss)
    torch.cuda.synchronize()
    dl = sign * f64(dw)[int(t[0]), 8:8 + T]
    assert dl.max() <= 0.0
    assert np.all(dl >= -1.01 * U32 * (np.abs(f64(lse)) + 16))


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_infinities_in_the_vocabulary_stay_as_the_formula_has_them(act):
    """A word at minus infinity takes no part; a token without a finite logit,
    or with one at infinity, has no finite loss."""
    h, w = torch.zeros(3, 64), torch.zeros(300, 64)
    h[:, 0] = torch.tensor([2.0, 4.0, -1.0])
    w[:, 0] = -0.5
    w[250, 0] = -float("inf")
    t = torch.tensor([7, 8, 9], device="cuda")
    loss, lse = model.vocab_loss(h.to(DTYPES[act]).cuda(), w.to(DTYPES[act]).cuda(), t)
    torch.cuda.synchronize()
    want = np.log(299.0)
    within("loss", loss[:2], np.array([want, want]), 200 * U32)
    within("lse", lse[:2], np.array([want - 1.0, want - 2.0]), 200 * U32)
    assert not torch.isfinite(loss[2]) and not torch.isfinite(lse[2])


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("at", ["largest", "other"])
def test_logits_of_any_size(at, act):
    """Logits from 2^31 to 2^90, whose steps in float32 are themselves large: the
    loss is the difference to the largest, rounded once, and 0 for the largest;
    a sure token's gradient is 0, a wrong one's -g at the target and g at the
    largest."""
    rng = np.random.default_rng(8)
    T, V, d = 60, 700, 72
    h, w = torch.zeros(T, d), torch.zeros(V, d)
    h[:, 0] = _bf16(rng.uniform(1.0, 2.0, T)) * 2.0 ** torch.linspace(31, 90, T).round()
    h[range(T), range(8, 8 + T)] = 1.0
    w[:, 0] = _bf16(rng.uniform(-1.0, 0.0, V))
    w[411, 0] = 1.25
    t = torch.full((T,), 411 if at == "largest" else 17, dtype=torch.int64, device="cuda")
    h, w = h.to(DTYPES[act]).cuda(), w.to(DTYPES[act]).cuda()
    loss, lse = model.vocab_loss(h, w, t)
    _, dw = model.vocab_loss_backward(h, w, t, lse, torch.ones(T, device="cuda"))
    torch.cuda.synchronize()
    L = f64(h)[:, 0] * 1.25
    within("lse", lse, L, U32 * L)
    within("loss", loss, L - f64(h)[:, 0] * f64(w)[int(t[0]), 0], 2 * U32 * L if at == "other" else 0.0)
    dl = f64(dw)[:, 8:8 + T]
    want = np.zeros((V, T))
    if at == "other":
        want[411], want[17] = 1.0, -1.0
    assert np.array_equal(dl, want)
