"""Clipping by factors below float32's smallest normal number, 1.2e-38: gradients of up to 1e38
with bounds far under 1. The factor keeps its 24 bits, the scaled values are off by the
factor's and their own rounding, as in any other case."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from model_cases import DTYPES, U16, U32, f64, within  # noqa: E402
from oracle import model_oracle as M  # noqa: E402
from orthogonal_equivalence_amd import model  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible AMD GPU"
    torch.cuda.init()


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("max_norm", [1.0, 0.5, 1e-3, 1e-7, 1e-12, 1e-30])
@pytest.mark.parametrize("offset", [0, 1])
def test_small_factors(offset, max_norm, act):
    rng = np.random.default_rng(3)
    size = [1e38, 1e30, 1e10, 1.0]
    grads = [torch.from_numpy((s * rng.uniform(-3, 3, n)).astype(np.float32)).to(DTYPES[act]).cuda()
             for s, n in zip(size, (1003, 50, 4099, 7))]
    NORM, OUT = M.clip_grad_norm([f64(g) for g in grads], max_norm)
    out = [torch.full((g.numel() + 1,), 7.0, dtype=g.dtype, device="cuda")[offset:offset + g.numel()] for g in grads]
    model.clip_grad_norm(grads, max_norm, out=out)
    model.clip_grad_norm(grads, max_norm)   # in place
    assert max_norm / NORM < 2.0 ** -126
    r = U16 if act == "bf16" else U32
    # half a step of float32's smallest numbers, of bfloat16's those of 2^-133
    least = 2.0 ** -134 if act == "bf16" else 2.0 ** -150
    for g, o, want in zip(grads, out, OUT):
        within("scaled", o, want, (r + 4 * U32) * np.abs(want) + 2 * least)
        assert torch.equal(g, o)
