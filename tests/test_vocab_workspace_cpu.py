"""Workspace of the vocabulary loss: a buffer of the size for T tokens serves
every smaller number of tokens, though the fastest plans of fewer can ask for
more. Sizes are checked on the host before the workspace pointer, which is null
here, so that nothing is ever launched: POETX_EWORKSPACE says too small,
POETX_EINVAL that the size was enough."""

import pytest

px = pytest.importorskip("orthogonal_equivalence_amd.poetx", reason="libpoetx.so not built")
from orthogonal_equivalence_amd import model_ops as mo  # noqa: E402

FAKE = 1 << 20


def enough(D, T, op, ws_bytes):
    with pytest.raises(px.PoetxError) as e:
        if op == mo.POETX_OP_VOCAB_FORWARD:
            mo.poetx_vocab_loss_forward(D, T, FAKE, D.d, FAKE, D.d, FAKE, FAKE, FAKE, None, ws_bytes, stream=0)
        else:
            mo.poetx_vocab_loss_backward(D, T, FAKE, D.d, FAKE, D.d, FAKE, FAKE, None, 1.0, FAKE, FAKE, None, ws_bytes,
                                         stream=0)
    assert e.value.status in (px.POETX_EWORKSPACE, px.POETX_EINVAL)
    return e.value.status == px.POETX_EINVAL


def _token_counts(most):
    """1, 2, .. to `most`, denser where tiles and pieces change."""
    out, t = [], 1
    while t < most:
        out += [t - 1, t, t + 1] if t > 1 else [1]
        t = max(t + 1, int(t * 1.07))
    return sorted({t for t in out if 0 < t <= most} | {most})


@pytest.mark.parametrize("op", [mo.POETX_OP_VOCAB_FORWARD, mo.POETX_OP_VOCAB_BACKWARD])
@pytest.mark.parametrize("d,V,dtype,piece", [(1024, 32000, "bf16", 0), (4096, 131072, "bf16", 0), (72, 200, "bf16", 0),
                                             (512, 1000, "f32", 0), (2056, 50021, "f32", 0), (64, 1 << 20, "bf16", 0),
                                             (1024, 32000, "bf16", 2048), (264, 700, "f32", 256)])
def test_a_workspace_serves_every_smaller_token_count(d, V, dtype, piece, op):
    D = mo.make_vocab(d, V, dtype, piece)
    counts = _token_counts(20000)
    sizes = [mo.poetx_vocab_ws_bytes(D, t, op) for t in counts]
    assert all(s > 0 for s in sizes)
    lower = [i for i, s in enumerate(sizes) if s < max(sizes[:i + 1])]  # the sizes below an earlier one
    for i in lower + [len(counts) - 1]:
        for t in counts[:i + 1]:
            assert enough(D, t, op, sizes[i]), (t, counts[i], sizes[i])


def test_the_sizes_do_fall_with_more_tokens():
    """What the test above is about: the switch points of the plans."""
    size = lambda d, V, T: mo.poetx_vocab_ws_bytes(mo.make_vocab(d, V), T, mo.POETX_OP_VOCAB_BACKWARD)  # noqa: E731
    assert size(1024, 32000, 4192) > size(1024, 32000, 4200)
    assert size(4096, 131072, 1736) > size(4096, 131072, 3072)


@pytest.mark.parametrize("op", [mo.POETX_OP_VOCAB_FORWARD, mo.POETX_OP_VOCAB_BACKWARD])
@pytest.mark.parametrize("piece", [0, 512])
def test_too_little_is_refused(op, piece):
    D = mo.make_vocab(264, 3001, piece=piece)
    T = 300
    have = mo.poetx_vocab_ws_bytes(D, T, op)
    assert enough(D, T, op, have) and not enough(D, T, op, 0)
    low, high = 0, have
    while high - low > 1:
        mid = (low + high) // 2
        low, high = (low, mid) if enough(D, T, op, mid) else (mid, high)
    # every part that no plan does without: gathered rows, indices, and a piece of 256 words with
    # dh's sums, or a pair per 256 columns
    least = T * 264 * 2 + 3 * T * 4
    least += T * 256 * 2 + T * 264 * 4 if op == mo.POETX_OP_VOCAB_BACKWARD else T * 12 * 8
    assert least <= high <= have
    for size in range(0, have, max(1, have // 97)):
        assert enough(D, T, op, size) == (size >= high)


@pytest.mark.parametrize("T", [131072, 131073, 400000, 1 << 20, 1 << 24])
@pytest.mark.parametrize("dtype,es", [("bf16", 2), ("f32", 4)])
def test_a_piece_of_very_many_tokens_holds_1024_words(T, dtype, es):
    """As documented: 256 MB a piece, but 1024 words where they take more (less up
    to a tenth where the pieces are evened out); beside it the gathered rows, dh's
    float sums, five values a token, and dw's sums where they are split."""
    d, V = 512, 32000
    size = mo.poetx_vocab_ws_bytes(mo.make_vocab(d, V, dtype), T, mo.POETX_OP_VOCAB_BACKWARD)
    parts = T * d * (es + 4) + 20 * T
    assert max(1 << 28, T * 1024 * es) * 0.9 + parts <= size <= max(1 << 28, T * 1024 * es) + parts + (1 << 28)
    asked = mo.poetx_vocab_ws_bytes(mo.make_vocab(d, V, dtype, 256), T, mo.POETX_OP_VOCAB_BACKWARD)
    assert T * 256 * es + parts <= asked <= T * 256 * es + parts + (1 << 28)
