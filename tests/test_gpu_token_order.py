"""The order of the alternatives where a group of neighbouring words holds a logit far
above the others: the logits there are kept as 16 bits of their distance below it, and
what these are bounds of has to hold for every float.

Rows of h are multiples of one unit vector, so that every logit is one product, exact in
float64, and rounded once in float32."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from model_cases import DTYPES, f64  # noqa: E402
from oracle import model_oracle as M  # noqa: E402
from orthogonal_equivalence_amd import model  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible AMD GPU"
    torch.cuda.init()


def _check(values, act, top, T=1):
    """The alternatives of words whose logits are the values (and twice, three times .. them
    in the other rows: powers of two, to keep them exact)."""
    V = len(values)
    w = torch.zeros((V, 64), dtype=DTYPES[act], device="cuda")
    w[:, 5] = torch.from_numpy(np.asarray(values, np.float32)).to(DTYPES[act]).cuda()
    h = torch.zeros((T, 64), dtype=DTYPES[act], device="cuda")
    h[:, 5] = 2.0 ** (torch.arange(T, device="cuda") % 3)
    _, _, _, ids, alt = model.token_logprobs(h, w, top=top)
    L = f64(h)[:, 5:6] * f64(w)[None, :, 5]
    want = M.top_tokens(L, np.ones(T, bool), top)[0]
    bad = np.flatnonzero((ids.cpu().numpy() != want).any(1))
    assert bad.size == 0, (bad[:5], ids[bad[0]].tolist(), want[bad[0]].tolist())


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 300, 600])
def test_words_near_0_beside_a_large_one(T, act):
    """1e-6 - 100 is -100 in float32: the distance is rounded up, the logit is not 0."""
    print(f"\n[gpu] order near 0 T={T} {act}", flush=True)
    values = np.full(4000, -5.0)
    values[0], values[1], values[32::32] = 100.0, 1e-6, 1e-6
    _check(values, act, 5, T)
    values[0], values[1] = 9984.0, 2e-6
    _check(values, act, 5, T)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("V", [200, 3000, 20000])
def test_small_logits_in_the_groups_of_large_ones(V, seed, act):
    """A few groups with a large logit hold the largest of the small ones, too."""
    print(f"\n[gpu] order of small logits V={V} seed={seed} {act}", flush=True)
    rng = np.random.default_rng([V, seed])
    small = 10.0 ** rng.uniform(-9, -1)
    values = small * rng.random(V)
    at = rng.permutation(V // 64)[:3] * 64
    values[at + rng.integers(0, 8)] = rng.uniform(50, 30000, 3)
    values[at + 8] = small * (1 + np.arange(3) / 8)
    values[at + 9] = small * 1.0625
    _check(values, act, 6)
    _check(values - small, act, 6)   # beside 0 on the other side
