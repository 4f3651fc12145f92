"""The vocabulary loss under every plan of its sums: the fastest one, those of a
smaller workspace, and splits behind wide tiles; errors of whole matrices
against the float64 form.

Bound of ||got - want|| / ||want|| for dh and dw, in bfloat16: every term dl and
every output is rounded to 8 bits on its own, an error spread evenly over half a
step, at most 2^-8 / sqrt(3) of a value in the root mean square; the terms of a
sum add like the errors of independent values, so that two such roundings make
sqrt(2 / 3) 2^-8 = 0.32% at most. float32 sums are off by less than 1e-4 of
that. In float32: a logit is off by (d / 2 + 2) u32 times sum |h w|, dl by as
much relative, twice with lse's own.
"""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from model_cases import U16, U32, f64, normal  # noqa: E402
from oracle import model_oracle as M  # noqa: E402
from orthogonal_equivalence_amd import model  # noqa: E402
from orthogonal_equivalence_amd import model_ops as mo  # noqa: E402
from orthogonal_equivalence_amd import poetx as px  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible AMD GPU"
    torch.cuda.init()


def _inputs(rng, T, d, V, act, ignored):
    h, w = normal(rng, (T, d), act), normal(rng, (V, d), act, 2.0 / np.sqrt(d))
    t = rng.integers(0, V, T)
    t[rng.random(T) < ignored] = -100
    return h, w, torch.from_numpy(t).cuda()


def _bound(h, w, act):
    if act == "bf16":
        return np.sqrt(2.0 / 3.0) * U16
    most = float((h.abs() @ w.abs().t()).max())
    return 4 * (h.shape[1] / 2 + 2) * U32 * most


def _near(name, got, want, bound):
    off = np.linalg.norm(f64(got) - want) / np.linalg.norm(want)
    assert off <= bound, f"{name}: off by {off:.5f} of its size, bound {bound:.5f}"


def _want(h, w, t):
    counted = ((t >= 0) & (t < w.shape[0])).cpu().numpy()
    g = np.full(len(counted), 1.0 / max(1, counted.sum()))
    loss, lse, _ = M.vocab_loss(f64(h), f64(w), t.cpu().numpy())
    dh, dw, _ = M.vocab_loss_backward(f64(h), f64(w), t.cpu().numpy(), g)
    return loss, lse, dh, dw


def _guarded(size):
    """A workspace of `size` bytes, all ones (NaN as any float), and the guard behind it."""
    whole = torch.full((size + 4096,), 255, dtype=torch.uint8, device="cuda")
    return whole[:size], whole[size:]


def _enough(D, T, op, ws_bytes):
    """Whether the entry point takes that much, asked without a workspace: nothing is launched."""
    at = 1 << 20
    args = (D, T, at, D.d, at, D.d, at) + ((at, at) if op == mo.POETX_OP_VOCAB_FORWARD else (at, None, 1.0, at, at))
    f = mo.poetx_vocab_loss_forward if op == mo.POETX_OP_VOCAB_FORWARD else mo.poetx_vocab_loss_backward
    with pytest.raises(px.PoetxError) as e:
        f(*args, None, ws_bytes, stream=0)
    return e.value.status == px.POETX_EINVAL


def _least(D, T, op):
    low, high = 0, mo.poetx_vocab_ws_bytes(D, T, op)
    while high - low > 1:
        mid = (low + high) // 2
        low, high = (low, mid) if _enough(D, T, op, mid) else (mid, high)
    return high


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,V,ignored", [(70, 264, 9000, 0.2), (300, 136, 3001, 0.5), (1500, 72, 700, 0.0),
                                           (1, 64, 5000, 0.0)])
def test_smaller_workspaces(T, d, V, ignored, act):
    rng = np.random.default_rng([T, V])
    h, w, t = _inputs(rng, T, d, V, act, ignored)
    LOSS, LSE, DH, DW = _want(h, w, t)
    D = mo.make_vocab(d, V, act)
    F, B = mo.POETX_OP_VOCAB_FORWARD, mo.POETX_OP_VOCAB_BACKWARD
    full_f, full_b = (mo.poetx_vocab_ws_bytes(D, T, op) for op in (F, B))
    least_f, least_b = _least(D, T, F), _least(D, T, B)
    bound = _bound(h, w, act)
    for share in (0.0, 0.1, 0.3, 0.6, 0.9, 1.0):
        size_f, size_b = (int(lo + share * (hi - lo)) for lo, hi in ((least_f, full_f), (least_b, full_b)))
        print(f"\n[gpu] vocab_loss T={T} d={d} V={V} {act} workspaces {size_f} {size_b}", end="", flush=True)
        loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        ws, guard = _guarded(size_f)
        mo.poetx_vocab_loss_forward(D, T, h, d, w, d, t, loss, lse, ws, size_f)
        dh, dw = torch.empty_like(h), torch.empty_like(w)
        ws_b, guard_b = _guarded(size_b)
        mo.poetx_vocab_loss_backward(D, T, h, d, w, d, t, lse, None, 1.0, dh, dw, ws_b, size_b)
        torch.cuda.synchronize()
        assert torch.all(guard == 255) and torch.all(guard_b == 255)
        _near("loss", loss, LOSS, 1e-4)
        _near("lse", lse, LSE, 1e-4)
        _near("dh", dh, DH, bound)
        _near("dw", dw, DW, bound)


def test_the_workspace_of_more_tokens_serves_fewer():
    """Scratch sized once for the largest batch: the last batch's own plan asks for more."""
    d, V, most, T = 1024, 32000, 4200, 4192
    D, B = mo.make_vocab(d, V), mo.POETX_OP_VOCAB_BACKWARD
    size = mo.poetx_vocab_ws_bytes(D, most, B)
    assert size < mo.poetx_vocab_ws_bytes(D, T, B)
    print(f"\n[gpu] vocab_loss T={T} d={d} V={V} workspace {size}", flush=True)
    rng = np.random.default_rng(1)
    h, w = normal(rng, (T, d), "bf16"), normal(rng, (V, d), "bf16", 2.0 / np.sqrt(d))
    t = torch.from_numpy(rng.integers(0, V, T)).cuda()
    _, lse = model.vocab_loss(h, w, t)
    want = model.vocab_loss_backward(h, w, t, lse)
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    ws, guard = _guarded(size)
    mo.poetx_vocab_loss_backward(D, T, h, d, w, d, t, lse, None, 1.0, dh, dw, ws, size)
    torch.cuda.synchronize()
    assert torch.all(guard == 255)
    # both are within the bound of the same gradients
    _near("dh", dh, f64(want[0]), 2 * np.sqrt(2.0 / 3.0) * U16)
    _near("dw", dw, f64(want[1]), 2 * np.sqrt(2.0 / 3.0) * U16)


# rows, columns, workgroups at a time and cost of a round of the bfloat16 tiles, as the launcher has them
TILES = [(64, 64, 256, 11.2), (64, 64, 512, 16.8), (128, 128, 256, 22.0), (128, 256, 256, 35.0), (192, 256, 256, 46.5),
         (256, 256, 256, 57.0)]


def _k_plan(rows, cols, k, without=None):
    """Tile and splits of a bfloat16 product, by the launcher's rule."""
    steps, best, least = -(-k // 64), None, np.inf
    for i, (bm, bn, slots, us) in enumerate(TILES):
        if i == without:
            continue
        n = -(-rows // bm) * -(-cols // bn)
        for s in range(1, 17):
            if s > 1 and (steps < 8 * s or n * s > 4 * slots):
                break
            cost = -(-n * s // slots) * -(-steps // s) * us / 32
            cost += 4.0 + rows * cols * 8.0 * s / 4e6 if s > 1 else 0.0
            if cost < least:
                least, best = cost, (i, s)
    return best


# dh in every wide tile (its index in TILES) with a split of its sum over the
# vocabulary, with all and with some of the tokens counted, in one piece and in
# several whose sums add up
@pytest.mark.parametrize("ignored", [0.0, 0.6])
@pytest.mark.parametrize("T,d,V,piece,plan", [(1000, 1536, 6000, 0, (3, 5)), (1500, 1536, 12000, 0, (4, 5)),
                                              (1200, 2504, 8000, 0, (5, 5)), (1000, 2504, 9000, 4096, (3, 3)),
                                              (1200, 2048, 16100, 8192, (3, 3)), (1200, 2504, 16384, 8192, (5, 5))])
def test_wide_tiles_with_a_split_sum(T, d, V, piece, plan, ignored):
    words = min(piece or V, V)
    assert _k_plan(T, d, words) == plan
    # the library's splits show in the size of its sums
    splits_w = _k_plan(words, d, T, without=4)[1]
    sums = 4 * d * (plan[1] * T + (splits_w * words if splits_w > 1 else 0))
    size = mo.poetx_vocab_ws_bytes(mo.make_vocab(d, V, "bf16", piece), T, mo.POETX_OP_VOCAB_BACKWARD)
    rest = size - sums - 2 * T * (-(-words // 256) * 256 + -(-d // 64) * 64)
    assert 0 < rest < 64 * T
    print(f"\n[gpu] vocab_loss T={T} d={d} V={V} piece={piece} ignored={ignored}", flush=True)
    rng = np.random.default_rng([T, d, V, int(10 * ignored)])
    h, w, t = _inputs(rng, T, d, V, "bf16", ignored)
    LOSS, LSE, DH, DW = _want(h, w, t)
    loss, lse = model.vocab_loss(h, w, t, piece)
    dh, dw = model.vocab_loss_backward(h, w, t, lse, piece=piece)
    torch.cuda.synchronize()
    bound = _bound(h, w, "bf16")
    _near("loss", loss, LOSS, 1e-4)
    _near("lse", lse, LSE, 1e-4)
    _near("dh", dh, DH, bound)
    _near("dw", dw, DW, bound)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,V,counted", [(255, 264, 3001, 255), (600, 136, 500, 255), (260, 512, 2000, 255),
                                           (700, 128, 5000, 510)])
def test_errors_of_whole_matrices(T, d, V, counted, act):
    """The mean loss over 255 or 510 tokens: 1 / 255 lies almost half a step of
    bfloat16 from its neighbours, so that a factor rounded into the targets'
    terms, all alike, is an error of 0.39% by itself, outside the bound."""
    print(f"\n[gpu] vocab_loss T={T} d={d} V={V} counted={counted} {act}", flush=True)
    rng = np.random.default_rng([T, counted])
    h, w, t = _inputs(rng, T, d, V, act, 0.0)
    t[torch.from_numpy(rng.permutation(T)[counted:]).cuda()] = -100
    _, _, DH, DW = _want(h, w, t)
    _, lse = model.vocab_loss(h, w, t)
    dh, dw = model.vocab_loss_backward(h, w, t, lse)
    torch.cuda.synchronize()
    bound = _bound(h, w, act)
    _near("dh", dh, DH, bound)
    _near("dw", dw, DW, bound)
