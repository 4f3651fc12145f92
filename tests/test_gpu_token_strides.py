"""Log probabilities of rows that lie far apart, such as the last tokens of long
sequences: a row every 2^22 elements or more, which is past what the offsets of a
tile's rows span. The results are those of the same rows side by side, bit for bit:
every row's sums are taken in the same order."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from model_cases import DTYPES, normal  # noqa: E402
from orthogonal_equivalence_amd import model  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible AMD GPU"
    torch.cuda.init()


def _apart(h, stride):
    """The same rows, `stride` elements from one to the next. What lies between them is
    whatever memory held."""
    far = torch.empty((h.shape[0] - 1) * stride + h.shape[1], dtype=h.dtype, device="cuda")
    far = far.as_strided(h.shape, (stride, 1))
    far.copy_(h)
    return far


# the last of a tile's rows past 2^31 bytes, and past 2^32, where 32-bit offsets start again
@pytest.mark.parametrize("act,stride", [("bf16", 1 << 22), ("bf16", (1 << 22) + 64), ("bf16", 1 << 24), ("f32", 1 << 22),
                                        ("f32", (1 << 22) + 64), ("f32", 1 << 24)])
@pytest.mark.parametrize("T,V,top,given", [(300, 900, 5, False), (300, 900, 0, False), (300, 900, 5, True), (270, 20000, 3, False),
                                           (270, 20000, 0, True), (140, 50021, 4, True), (600, 50021, 0, False)])
def test_rows_far_apart(T, V, top, given, act, stride):
    print(f"\n[gpu] token strides T={T} V={V} top={top} given={given} {act} ldh={stride}", flush=True)
    rng = np.random.default_rng(V)
    h, w = normal(rng, (T, 72), act), normal(rng, (V, 72), act, 0.3)
    t = torch.from_numpy(rng.integers(-V // 5, V, T)).cuda() if given else None
    far = _apart(h, stride)
    assert far.stride(0) == stride and far.dtype == DTYPES[act]
    want, got = model.token_logprobs(h, w, t, top=top), model.token_logprobs(far, w, t, top=top)
    da = normal(rng, T, "f32") if given else None
    db = normal(rng, T, "f32")
    want += model.token_logprobs_backward(h, w, t, want[2], want[1], da, db)
    got += model.token_logprobs_backward(far, w, t, got[2], got[1], da, db)
    torch.cuda.synchronize()
    for k, (a, b) in enumerate(zip(want, got)):
        assert (a is None and b is None) or torch.equal(a, b), k


def test_the_last_tokens_of_long_sequences():
    B, S, d, V = 128, 4096, 1024, 5000
    g = torch.Generator(device="cuda").manual_seed(4)
    hidden = torch.empty((B, S, d), dtype=torch.bfloat16, device="cuda")
    hidden[:, -1] = torch.randn((B, d), generator=g, device="cuda").bfloat16()
    w = (0.05 * torch.randn((V, d), generator=g, device="cuda")).bfloat16()
    want = model.token_logprobs(hidden[:, -1].contiguous(), w, top=5)
    got = model.token_logprobs(hidden[:, -1], w, top=5)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert (a is None and b is None) or torch.equal(a, b)
