"""Gradients of log probabilities under small and large temperatures: upstream gradients
and the factor 1 / temperature each fit float32, their product need not, and the gradients
still may.

Scaled by powers of two throughout, the logits over the temperature are the same bit for bit,
and so are the gradients but for their own power of two."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from model_cases import normal  # noqa: E402
from orthogonal_equivalence_amd import model  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible AMD GPU"
    torch.cuda.init()


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,piece", [(40, 300, 0), (40, 3000, 512), (5000, 100, 0), (64, 20000, 0)])
@pytest.mark.parametrize("size,up", [(-33, 70), (33, -70), (-20, 0), (30, 0)])
def test_powers_of_two(size, up, T, V, piece, act):
    """Rows of h and w times 2^size, the temperature times 2^(2 size), gradients times 2^up:
    gradients times 2^(up - size). For the first two the product of gradient and factor is
    2^136 and 2^-136."""
    print(f"\n[gpu] token scales T={T} V={V} size={size} up={up} {act}", flush=True)
    rng = np.random.default_rng([T, V])
    h, w = normal(rng, (T, 64), act), normal(rng, (V, 64), act, 0.25)
    t = torch.from_numpy(rng.integers(-V // 5, V, T)).cuda()
    a, b = normal(rng, T, "f32"), normal(rng, T, "f32")

    def run(h, w, a, b, tau):
        out = model.token_logprobs(h, w, t, top=3, temperature=tau)
        return out, model.token_logprobs_backward(h, w, t, out[2], out[1], a, b, tau, piece)

    want, grads = run(h, w, a, b, 0.75)
    s = 2.0 ** size
    got, scaled = run(h * s, w * s, a * 2.0 ** up, b * 2.0 ** up, 0.75 * s * s)
    torch.cuda.synchronize()
    for k in (0, 1, 3, 4):
        assert torch.equal(want[k], got[k]), k
    for x, y in zip(grads, scaled):
        assert torch.isfinite(y).all()
        # but for what lies below the smallest normal number, where it is rounded in other places
        assert torch.allclose(x.double() * 2.0 ** (up - size), y.double(), rtol=0, atol=2.0 ** -125)
        if up >= 0:
            big = x.double().abs() > 2.0 ** -60
            assert torch.equal((x.double() * 2.0 ** (up - size))[big], y.double()[big])


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_the_smallest_temperature(act):
    """Every row is sure of its largest logit: no gradient, whatever the factors."""
    rng = np.random.default_rng(5)
    h, w = normal(rng, (30, 64), act), normal(rng, (200, 64), act, 0.25)
    t = (h.float() @ w.float().t()).argmax(1)
    a = torch.full((30,), 1e3, device="cuda")
    logprob, entropy, stat, ids, alt = model.token_logprobs(h, w, t, top=1, temperature=4.24e-39)
    dh, dw = model.token_logprobs_backward(h, w, t, stat, entropy, a, a, 4.24e-39)
    torch.cuda.synchronize()
    assert torch.equal(ids[:, 0], t)
    for x in (logprob, entropy, alt, dh, dw):
        assert torch.all(x == 0)
