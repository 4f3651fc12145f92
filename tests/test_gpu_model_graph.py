"""The operators around the layer captured in a HIP graph and replayed: every
replay gives what an eager pass gives, also with eager work and
synchronisations between the replays and with new inputs in place of the
captured ones."""

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


def _replays(make, step):
    """make(seed) -> input tensors; step(*inputs) -> output tensors."""
    static = make(0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            step(*static)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*static)
    for seed in (1, 2, 3, 2):
        new = make(seed)
        for a, b in zip(static, new):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        want = step(*new)
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w), seed


def test_norm_and_int8_product():
    def make(seed):
        rng = np.random.default_rng(seed)
        wt = torch.from_numpy(rng.integers(-127, 128, (784, 512)).astype(np.int8)).cuda()
        return [normal(rng, (40, 512), "bf16"), normal(rng, (40, 512), "bf16"), normal(rng, 512, "f32"), wt,
                normal(rng, 784, "f32").abs()]

    def step(x, r, gain, wt, scale):
        h, q, qs = model.rms_norm_q8(x, gain, r)
        return h, model.linear_i8(q, qs, wt, scale), model.linear_i8(q[:3], qs[:3], wt, scale)

    print("\n[gpu] graph: norm to int8 rows, int8 product", flush=True)
    _replays(make, step)


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_norm_and_loss_with_their_gradients(act):
    def make(seed):
        rng = np.random.default_rng(seed)
        t = torch.from_numpy(rng.integers(-30, 900, 300)).cuda()   # another number counted each time
        return [normal(rng, (300, 256), act), normal(rng, 256, "f32"), normal(rng, (900, 256), act, 0.1), t]

    def step(x, gain, w, t):
        h, y, rstd = model.rms_norm(x, gain, x)
        loss, lse = model.vocab_loss(y, w, t)
        dy, dw = model.vocab_loss_backward(y, w, t, lse, piece=512)
        dx, dgain = model.rms_norm_backward(dy, h, rstd, gain)
        return loss, dw, dx, dgain

    print(f"\n[gpu] graph: norm and vocabulary loss {act}", flush=True)
    _replays(make, step)
