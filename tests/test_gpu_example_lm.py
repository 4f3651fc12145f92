"""The operators and the layer together: the small language model of
``example_lm`` trains, its gradients agree with differences of its loss, and
its int8 serving path agrees with the layers it was exported from."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from orthogonal_equivalence_amd import example_lm, model  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible AMD GPU"
    torch.cuda.init()


def test_trains_merges_and_serves():
    losses, trained, served = example_lm.train(steps=40, interval=20, say=lambda s: print("[gpu] " + s, flush=True))
    # nine in ten successors are fixed: from log(1000) = 6.9 towards 0.33 + 0.1 log(1000) = 1.0
    assert losses[0] > 6.0 and losses[-1] < 0.8 * losses[0]
    # int8 rows are uniform in steps of max / 127: under 1% of a row, two layers deep
    assert abs(trained - served) < 0.02 * trained


def test_gradients_of_the_whole_step_against_differences():
    lm = example_lm.TinyLM(vocab=300, width=128, blocks=2, block_size=64, T_max=96)
    tokens, target = example_lm.batch(300, 96, 5)
    _, grads = lm.step(tokens, target)

    def loss():
        return float(lm.step(tokens, target)[0])

    # along each gain's and each rotation's gradient the loss has to change by
    # its squared norm; the activations' bfloat16 rounding (2^-9 of each, one
    # in ~100 rows' worth of the mean) is well under a tenth of these steps
    for p, g in zip(lm.parameters()[:-1], grads[:-1]):
        norm = float(g.double().norm())
        if norm == 0:
            continue
        d = g / norm
        step = min(0.1 / norm, 0.5 if p.numel() == 128 else 0.05)
        base = p.clone()
        p.copy_(base + step * d)
        up = loss()
        p.copy_(base - step * d)
        down = loss()
        p.copy_(base)
        assert (up - down) / (2 * step) == pytest.approx(norm, rel=0.15), (p.shape, step)


def test_one_token_serving_matches_a_batch():
    lm = example_lm.TinyLM(vocab=300, width=256, blocks=2, block_size=128, T_max=64)
    lm.merge(1)
    weights = lm.export()
    tokens, _ = example_lm.batch(300, 64, 6)
    rows = lm.serve(weights, tokens)
    for t in (0, 17, 63):
        one = lm.serve(weights, tokens[t:t + 1])
        assert torch.equal(one[0], rows[t])   # rows are independent, and the integer sums exact
    loss, _ = model.vocab_loss(rows, lm.w, tokens)
    assert torch.isfinite(loss).all()
