"""Alternatives where more words could be among them, by the 16 bits that are held of
each logit, than are ordered at a time: groups of neighbouring words with a logit far above
the others, whose bits say little about the rest of the group; finely rising logits; and
words that are equal in whole or in part.

Rows of h are multiples of one unit vector: every logit is one product, exact in float64 and
in float32."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_token_order import _check, _gpu  # noqa: E402, F401


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 300, 600])
@pytest.mark.parametrize("size", [1000, 30000])
@pytest.mark.parametrize("V,groups,top", [(8000, 12, 20), (8000, 20, 40), (8000, 55, 64), (40000, 30, 64), (2500, 20, 30)])
def test_outliers_in_groups_of_their_own(V, groups, top, size, T, act):
    """The words behind the outliers lie in other groups than theirs, at the other end."""
    print(f"\n[gpu] outliers V={V} in {groups} groups, top={top} of {size} T={T} {act}", flush=True)
    rng = np.random.default_rng([V, groups])
    values = rng.standard_normal(V)
    at = np.arange(min(groups, V // 64)) * 64
    values[at + rng.integers(0, 32, len(at))] = size * rng.uniform(0.9, 1.1, len(at))
    values[V - 2 * top:] += 2.0
    _check(values, act, top, T)
    _check(values[::-1].copy(), act, top, T)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 300, 600])
def test_equal_words_beside_outliers(T, act):
    """Thousands of equal logits, in the groups of outliers and in others; larger ones behind
    the first 512 of them."""
    print(f"\n[gpu] outliers and equal words T={T} {act}", flush=True)
    rng = np.random.default_rng(T)
    values = np.zeros(9000)
    values[np.arange(10) * 64 + 3] = rng.uniform(500, 1500, 10)
    _check(values, act, 20, T)
    values[6000:6005] = 0.25 * (1 + np.arange(5))
    _check(values, act, 20, T)
    _check(values, act, 12, T)
    values[700:8000] = 0.125
    _check(values, act, 64, T)
    values[8990] = 0.5
    _check(values, act, 20, T)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 300, 600])
@pytest.mark.parametrize("step", [2.0 ** -30, 1.0])
def test_whole_groups_of_few_values(step, T, act):
    """Every group alike, or rising from group to group in steps of few bits."""
    print(f"\n[gpu] alike groups T={T} step={step} {act}", flush=True)
    k = np.arange(12800)
    _check(k % 64 * step, act, 64, T)
    _check(k // 64 % 128 * step, act, 64, T)
    _check((k // 64 % 128 + 128) * step, act, 50, T)
    _check(-(k % 7) * step, act, 30, T)
    _check(np.where(k % 32 == 5, 100.0, -(k % 32) * step), act, 64, T)
