"""The float64 forms of the operators around the layer against differences of
their own losses and against cases with known values."""

import numpy as np
import pytest

from oracle import model_oracle as M


def _diff(f, x, d, h=1e-6):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


def test_norm_gradients_against_differences():
    rng = np.random.default_rng(0)
    x, r, g = rng.normal(size=(5, 24)), rng.normal(size=(5, 24)), rng.normal(size=24)
    dy, dh = rng.normal(size=(5, 24)), rng.normal(size=(5, 24))

    def loss(x_, g_):
        h, y, _ = M.rms_norm(x_, g_, r, 1e-3)
        return np.sum(dy * y) + np.sum(dh * h)

    h, _, rstd = M.rms_norm(x, g, r, 1e-3)
    dx, dg = M.rms_norm_backward(dy, h, g, 1e-3, dh)
    dx2, _ = M.rms_norm_backward(dy, h, g, 1e-3, dh, rstd)
    assert np.allclose(dx, dx2, rtol=1e-13)
    for _ in range(8):
        v, w = rng.normal(size=x.shape), rng.normal(size=g.shape)
        assert _diff(lambda a: loss(a, g), x, v) == pytest.approx(np.sum(dx * v), rel=1e-7, abs=1e-7)
        assert _diff(lambda a: loss(x, a), g, w) == pytest.approx(np.sum(dg * w), rel=1e-7, abs=1e-7)


def test_norm_known_values():
    _, y, rstd = M.rms_norm([[3.0, 4.0, 0.0, 0.0]], np.array([1.0, 2.0, 1.0, 1.0]), eps=0.0)
    assert rstd[0] == pytest.approx(0.4) and np.allclose(y, [[1.2, 3.2, 0, 0]])
    _, y, _ = M.rms_norm(np.zeros((2, 8)), np.ones(8), eps=1e-6)
    assert np.all(y == 0)


def test_quantised_rows_known_values():
    q, s = M.quantize_rows([[127.0, -63.5, 0.4, 1.5], [0, 0, 0, 0], [-254.0, 3.0, 5.0, 1.0]])
    assert s.tolist() == [1.0, 1.0, 2.0]
    assert q.tolist() == [[127, -64, 0, 2], [0, 0, 0, 0], [-127, 2, 2, 0]]  # ties to even


def test_vocab_gradients_against_differences():
    rng = np.random.default_rng(1)
    h, w = rng.normal(size=(6, 8)), rng.normal(size=(11, 8))
    t, g = np.array([3, -100, 10, 0, 11, 3]), rng.normal(size=6)
    loss = lambda h_, w_: np.sum(g * M.vocab_loss(h_, w_, t)[0])  # noqa: E731
    dh, dw, dl = M.vocab_loss_backward(h, w, t, g)
    for _ in range(8):
        v, u = rng.normal(size=h.shape), rng.normal(size=w.shape)
        assert _diff(lambda a: loss(a, w), h, v) == pytest.approx(np.sum(dh * v), rel=1e-7, abs=1e-7)
        assert _diff(lambda a: loss(h, a), w, u) == pytest.approx(np.sum(dw * u), rel=1e-7, abs=1e-7)
    assert np.all(dh[[1, 4]] == 0) and np.all(dl[[1, 4]] == 0)


def test_vocab_known_values():
    loss, lse, counted = M.vocab_loss(np.zeros((3, 4)), np.ones((16, 4)), np.array([0, 15, 16]))
    assert np.allclose(loss, [np.log(16), np.log(16), 0]) and counted.tolist() == [True, True, False]
    loss, _, _ = M.vocab_loss(np.ones((2, 4)), np.ones((1, 4)), np.array([0, -1]))
    assert loss.tolist() == [0.0, 0.0]  # one word: certain


def test_vocab_rows_not_counted_are_never_read():
    h = np.ones((3, 4))
    h[1] = np.nan
    t = np.array([0, -100, 2])
    assert np.all(np.isfinite(M.vocab_loss(h, np.eye(4), t)[0]))
    dh, dw, _ = M.vocab_loss_backward(h, np.eye(4), t, np.ones(3))
    assert np.all(np.isfinite(dh)) and np.all(np.isfinite(dw))


def test_linear_i8_known_values():
    xq, wt = np.array([[127, -127], [1, 2]]), np.array([[127, 127], [3, -1], [-127, 127]])
    z = M.linear_i8(xq, [0.5, 2.0], wt, [1.0, 10.0, 0.25])
    assert z.tolist() == [[0.0, 2540.0, -127 * 127 * 2 * 0.125], [762.0, 20.0, 63.5]]
