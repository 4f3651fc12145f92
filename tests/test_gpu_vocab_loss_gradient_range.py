"""The vocabulary loss's upstream gradients g[t] = scale * dloss[t] at the ends
of float32's range."""

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
@pytest.mark.parametrize("T", [20, 9000])
def test_a_gradient_that_the_scale_takes_past_the_range_stays_with_its_token(T, act):
    rng = np.random.default_rng(3)
    h, w = normal(rng, (T, 64), act), normal(rng, (300, 64), act)
    t = torch.from_numpy(rng.integers(0, 300, T)).cuda()
    _, lse = model.vocab_loss(h, w, t)
    dloss, scale = normal(rng, T, "f32"), 2.0 ** 100
    dloss[7] = 0
    want, _ = model.vocab_loss_backward(h, w, t, lse, dloss, scale)
    dloss[7] = 2.0 ** 40
    got, _ = model.vocab_loss_backward(h, w, t, lse, dloss, scale)
    torch.cuda.synchronize()
    keep = [i for i in range(T) if i != 7]
    assert torch.isfinite(want).all()
    assert torch.equal(got[keep], want[keep]) and not torch.isfinite(got[7]).any()


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [float("inf"), float("nan")])
def test_no_token_counted_adds_nothing_whatever_the_scale(scale, act):
    rng = np.random.default_rng(4)
    h, w = normal(rng, (40, 64), act), normal(rng, (300, 64), act)
    t = torch.full((40,), -100, dtype=torch.int64, device="cuda")
    _, lse = model.vocab_loss(h, w, t)
    for dloss in (None, torch.ones(40, device="cuda")):
        dh, dw = model.vocab_loss_backward(h, w, t, lse, dloss, scale)
        torch.cuda.synchronize()
        assert torch.all(dh == 0) and torch.all(dw == 0)
