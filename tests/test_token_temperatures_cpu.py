"""Temperatures of the log probabilities: the factor 1 / temperature has to be finite,
and with it the factor of the powers of two, log2(e) / temperature (the pointers are fake
and never used)."""

import numpy as np
import pytest

px = pytest.importorskip("orthogonal_equivalence_amd.poetx", reason="libpoetx.so not built")
from orthogonal_equivalence_amd import model_ops as mo  # noqa: E402

FAKE = 1 << 20
LEAST = 4.24e-39   # 1.442695 / 3.402823e38 is 4.2397e-39


def _statuses(tau):
    D = mo.make_vocab(64, 1000)
    calls = (lambda: mo.poetx_token_logprobs(D, 4, tau, FAKE, 64, FAKE, 64, FAKE, 0, FAKE, FAKE, FAKE, None, None, FAKE, 8, stream=0),
             lambda: mo.poetx_token_logprobs_backward(D, 4, tau, FAKE, 64, FAKE, 64, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE,
                                                      8, stream=0))
    out = []
    for call in calls:
        with pytest.raises(px.PoetxError) as e:
            call()
        out.append(e.value.status)
    return out


@pytest.mark.parametrize("tau", [2.95e-39, 3.5e-39, 4.23e-39, 2.0 ** -130, 1e-39, 1e-45, 0.0])
def test_too_small(tau):
    with np.errstate(over="ignore"):
        assert tau == 0 or not np.isfinite(np.float32(1.4426950408889634 / float(np.float32(tau))))
    assert _statuses(tau) == [px.POETX_EINVAL] * 2


@pytest.mark.parametrize("tau", [LEAST, 1.2e-38, 1e-30, 1.0, 3e38])
def test_taken(tau):
    # all checks passed but the last, the workspace's
    assert _statuses(tau) == [px.POETX_EWORKSPACE] * 2
