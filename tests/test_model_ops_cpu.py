"""Host-side checks of the operators around the layer (include/poetx_model.h):
every declared entry point is exported and bound, workspace sizes follow the
operators' plans, and invalid arguments are refused before any launch (fake
but aligned pointers are never dereferenced)."""

import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "poetx_model.h")

px = pytest.importorskip("orthogonal_equivalence_amd.poetx", reason="libpoetx.so not built")
from orthogonal_equivalence_amd import model_ops as mo  # noqa: E402

FAKE = 1 << 20
BF, F32 = px.POETX_BF16, px.POETX_F32


def _status(call):
    with pytest.raises(px.PoetxError) as e:
        call()
    return e.value.status


def test_every_declared_symbol_is_exported_and_bound():
    names = sorted(set(re.findall(r"POETX_API\s+[\w\s\*]+?\b(poetx_\w+)\s*\(", open(HEADER).read())))
    assert names == sorted(mo.EXPORTED) == sorted(mo._sig)
    for n in names:
        assert hasattr(px._lib, n) and callable(getattr(mo, n))


NORM = dict(T=4, n=64, dtype=BF, x=FAKE, ldx=64, res=2 * FAKE, ldr=64, gain=FAKE, eps=1e-6, h=3 * FAKE, out=4 * FAKE,
            aux=5 * FAKE)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("bad", [
    dict(n=0), dict(n=4), dict(n=60), dict(n=(1 << 24) + 16, ldx=(1 << 24) + 16, ldr=(1 << 24) + 16),
    dict(T=-1), dict(T=(1 << 30) + 1), dict(dtype=px.POETX_I8), dict(dtype=7),
    dict(ldx=56), dict(ldx=68), dict(ldr=63), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(x=None), dict(x=FAKE + 8), dict(res=FAKE + 2), dict(gain=None), dict(h=FAKE + 4), dict(out=None),
    dict(h=FAKE, ldx=128),               # in place needs contiguous rows
    dict(h=2 * FAKE, ldr=128),
])
def test_norm_refuses(bad, q8):
    a = {**NORM, **bad}
    f = mo.poetx_rmsnorm_forward_q8 if q8 else mo.poetx_rmsnorm_forward
    assert _status(lambda: f(a["T"], a["n"], a["dtype"], a["x"], a["ldx"], a["res"], a["ldr"], a["gain"], a["eps"],
                             a["h"], a["out"], a["aux"], stream=0)) == px.POETX_EINVAL


def test_norm_q8_rows_are_whole_16_byte_chunks():
    args = lambda n: (4, n, BF, FAKE, n, None, 0, FAKE, 1e-6, None, FAKE, FAKE)  # noqa: E731
    assert _status(lambda: mo.poetx_rmsnorm_forward_q8(*args(72), stream=0)) == px.POETX_EINVAL
    assert _status(lambda: mo.poetx_quantize_rows(4, 72, BF, FAKE, 72, FAKE, FAKE, stream=0)) == px.POETX_EINVAL
    assert _status(lambda: mo.poetx_quantize_rows(4, 64, BF, FAKE, 64, FAKE, None, stream=0)) == px.POETX_EINVAL


BWD = dict(T=4, n=64, dtype=BF, dy=FAKE, lddy=64, h=2 * FAKE, rstd=FAKE, gain=FAKE, dh=3 * FAKE, lddh=64, dx=4 * FAKE,
           dgain=FAKE, ws=FAKE, ws_bytes=1 << 20)


@pytest.mark.parametrize("bad,status", [
    (dict(n=12), px.POETX_EINVAL), (dict(T=-1), px.POETX_EINVAL), (dict(dtype=3), px.POETX_EINVAL),
    (dict(dy=None), px.POETX_EINVAL), (dict(h=None), px.POETX_EINVAL), (dict(rstd=None), px.POETX_EINVAL),
    (dict(dx=None), px.POETX_EINVAL), (dict(dh=FAKE + 8), px.POETX_EINVAL), (dict(dgain=FAKE + 4), px.POETX_EINVAL),
    (dict(lddy=60), px.POETX_EINVAL), (dict(lddh=68), px.POETX_EINVAL),
    (dict(dx=FAKE, lddy=128), px.POETX_EINVAL), (dict(dx=3 * FAKE, lddh=128), px.POETX_EINVAL),
    (dict(ws_bytes=16), px.POETX_EWORKSPACE), (dict(ws=None, ws_bytes=1 << 20), px.POETX_EINVAL),
])
def test_norm_backward_refuses(bad, status):
    a = {**BWD, **bad}
    assert _status(lambda: mo.poetx_rmsnorm_backward(*a.values(), stream=0)) == status


def test_norm_workspace_holds_a_row_per_group():
    assert mo.poetx_rmsnorm_ws_bytes(0, 64) == 0
    assert mo.poetx_rmsnorm_ws_bytes(3, 60) == 0
    assert mo.poetx_rmsnorm_ws_bytes(3, 64) == 3 * 64 * 4
    big = mo.poetx_rmsnorm_ws_bytes(1 << 30, 4096)
    assert 0 < big <= 1024 * 4096 * 4 and mo.poetx_rmsnorm_ws_bytes(1 << 20, 4096) == big


LIN = dict(T=4, m=64, n=32, out=BF, xq=FAKE, xs=FAKE, wt=FAKE, ws_=FAKE, z=FAKE, ldz=32)


@pytest.mark.parametrize("bad", [
    dict(m=8), dict(m=72), dict(n=24), dict(m=131072), dict(n=(1 << 24) + 16, ldz=(1 << 24) + 16), dict(T=-1),
    dict(T=(1 << 24) + 1), dict(out=px.POETX_I8), dict(xq=None), dict(xs=None), dict(wt=FAKE + 8), dict(ws_=None),
    dict(z=None), dict(ldz=24), dict(ldz=36),
])
def test_linear_i8_refuses(bad):
    a = {**LIN, **bad}
    assert _status(lambda: mo.poetx_linear_i8(*a.values(), stream=0)) == px.POETX_EINVAL


def test_linear_i8_width_limit_keeps_every_sum_in_31_bits():
    assert 131056 * 128 * 128 < 2 ** 31 <= 131072 * 128 * 128
    assert _status(lambda: mo.poetx_linear_i8_prepare(131072, 16, FAKE, FAKE, stream=0)) == px.POETX_EINVAL
    assert _status(lambda: mo.poetx_linear_i8_prepare(64, 32, FAKE, None, stream=0)) == px.POETX_EINVAL


@pytest.mark.parametrize("bad", [dict(d=4), dict(d=68), dict(d=(1 << 17) + 8), dict(V=0), dict(V=(1 << 24) + 1),
                                 dict(piece=-1)])
def test_vocab_descriptor_is_checked(bad):
    D = mo.make_vocab(**{**dict(d=64, V=100), **bad})
    for op in (mo.POETX_OP_VOCAB_FORWARD, mo.POETX_OP_VOCAB_BACKWARD):
        assert mo.poetx_vocab_ws_bytes(D, 4, op) == 0
    ld = max(64, D.d)
    assert _status(lambda: mo.poetx_vocab_loss_forward(D, 4, FAKE, ld, FAKE, ld, FAKE, FAKE, FAKE, FAKE, 1 << 60,
                                                       stream=0)) == px.POETX_EINVAL
    assert _status(lambda: mo.poetx_vocab_loss_backward(D, 4, FAKE, ld, FAKE, ld, FAKE, FAKE, None, 1.0, FAKE, FAKE,
                                                        FAKE, 1 << 60, stream=0)) == px.POETX_EINVAL


VOC = dict(T=4, h=FAKE, ldh=64, w=FAKE, ldw=64, target=FAKE, a=FAKE, b=FAKE, ws=FAKE, ws_bytes=1 << 60)


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), px.POETX_EINVAL), (dict(T=(1 << 24) + 1), px.POETX_EINVAL), (dict(h=None), px.POETX_EINVAL),
    (dict(ldh=56), px.POETX_EINVAL), (dict(ldw=66), px.POETX_EINVAL), (dict(w=FAKE + 2), px.POETX_EINVAL),
    (dict(ldw=(1 << 22) + 8), px.POETX_EUNSUPPORTED), (dict(target=None), px.POETX_EINVAL),
    (dict(a=None), px.POETX_EINVAL), (dict(ws_bytes=8), px.POETX_EWORKSPACE), (dict(ws=None), px.POETX_EINVAL),
])
def test_vocab_loss_refuses(bad, status):
    D = mo.make_vocab(64, 1000)
    a = {**VOC, **bad}
    common = (D, a["T"], a["h"], a["ldh"], a["w"], a["ldw"], a["target"])
    assert _status(lambda: mo.poetx_vocab_loss_forward(*common, a["a"], a["b"], a["ws"], a["ws_bytes"],
                                                       stream=0)) == status
    assert _status(lambda: mo.poetx_vocab_loss_backward(*common, FAKE, None, 1.0, a["a"], a["b"], a["ws"],
                                                        a["ws_bytes"], stream=0)) == status


def test_products_past_one_launch_are_refused():
    # 2^24 tokens by 2^24 outputs: 2^32 tiles
    assert _status(lambda: mo.poetx_linear_i8(1 << 24, 64, 1 << 24, BF, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 24,
                                              stream=0)) == px.POETX_EUNSUPPORTED
    D = mo.make_vocab(64, 1 << 24)
    args = (D, 1 << 24, FAKE, 64, FAKE, 64, FAKE)
    assert _status(lambda: mo.poetx_vocab_loss_forward(*args, FAKE, FAKE, FAKE, 1 << 62,
                                                       stream=0)) == px.POETX_EUNSUPPORTED
    assert _status(lambda: mo.poetx_vocab_loss_backward(*args, FAKE, None, 1.0, FAKE, FAKE, FAKE, 1 << 62,
                                                        stream=0)) == px.POETX_EUNSUPPORTED


def test_vocab_workspace_is_bounded_by_the_piece_not_the_logits():
    T, d, V = 8192, 4096, 131072
    bwd = mo.poetx_vocab_ws_bytes(mo.make_vocab(d, V), T, mo.POETX_OP_VOCAB_BACKWARD)
    # a piece of 256 MB, the gathered rows and the float sums of dh
    assert bwd < (1 << 28) + T * d * 6 + T * 64
    assert bwd < T * V * 2 / 4
    small = mo.poetx_vocab_ws_bytes(mo.make_vocab(d, V, piece=1000), T, mo.POETX_OP_VOCAB_BACKWARD)
    assert small < T * 1024 * 2 + T * d * 6 + T * 64
    assert mo.poetx_vocab_ws_bytes(mo.make_vocab(d, V), T, mo.POETX_OP_VOCAB_FORWARD) < T * V // 4
    assert mo.poetx_vocab_ws_bytes(mo.make_vocab(d, V), T, 2) == 0
