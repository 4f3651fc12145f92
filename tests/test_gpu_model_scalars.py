"""Scalars in the place of the operators' gradients are refused as any other
wrong shape."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from orthogonal_equivalence_amd import model  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible AMD GPU"
    torch.cuda.init()


def test_scalar_gradients():
    rows, one = torch.ones((4, 64), device="cuda"), torch.ones((), device="cuda")
    line, t = torch.ones(4, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    gain = torch.ones(64, device="cuda")
    with pytest.raises(ValueError, match="dloss"):
        model.vocab_loss_backward(rows, rows, t, line, one)
    with pytest.raises(ValueError, match="dy"):
        model.rms_norm_backward(one, rows, line, gain)
    with pytest.raises(ValueError, match="dh"):
        model.rms_norm_backward(rows, rows, line, gain, dh=one)
