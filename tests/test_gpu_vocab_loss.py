"""Softmax cross entropy over a vocabulary, and its gradients, against the
float64 form.

Bounds. A logit is a float32 sum of d products of the inputs' exact values in
d / 16 (bfloat16; d / 2 in float32) matrix steps: off by at most (d / 16 + 16)
u32 (d / 2 + 2) times sum |h w|. lse adds a few u32 of its size and of the
longest chain of additions (32 columns, 4 waves, every 16th tile). dl is then
off by that much relative, plus u16 where it is rounded to bfloat16, and the
outputs by as much of sum |dl| |w| (sum |dl| |h|), plus their own rounding.
"""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from model_cases import U16, U32, f64, normal, strided, within  # noqa: E402
from oracle import model_oracle as M  # noqa: E402
from orthogonal_equivalence_amd import model  # noqa: E402
from orthogonal_equivalence_amd import poetx as px  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible AMD GPU"
    torch.cuda.init()


def _targets(rng, T, V, ignored):
    t = rng.integers(0, V, T)
    skip = rng.random(T) < ignored
    t[skip] = rng.choice([-100, -1, V, V + 7, 1 << 40], skip.sum())
    return torch.from_numpy(t).cuda()


def _check(h, w, t, act, dloss=None, scale=1.0, piece=0):
    H, W, N = f64(h), f64(w), t.cpu().numpy()
    T, d = H.shape
    loss, lse = model.vocab_loss(h, w, t, piece)
    dh, dw = model.vocab_loss_backward(h, w, t, lse, dloss, scale, piece)
    torch.cuda.synchronize()
    LOSS, LSE, counted = M.vocab_loss(H, W, N)
    sums = np.zeros(T)
    steps = d / 16 + 16 if act == "bf16" else d / 2 + 2
    if counted.any():
        sums[counted] = np.max(np.abs(H[counted]) @ np.abs(W).T, axis=1)
    off = steps * U32 * sums + (80 + W.shape[0] / 4096) * U32 + 4 * U32 * np.abs(LSE)
    within("lse", lse, LSE, off)
    within("loss", loss, LOSS, 2 * off)
    g = scale * (f64(dloss) if dloss is not None else np.full(T, 1.0 / max(1, counted.sum())))
    DH, DW, DL = M.vocab_loss_backward(H, W, N, g)
    r16 = U16 if act == "bf16" else 0.0
    # |dl| as it is composed: g (p + [v = target])
    size = np.abs(DL)
    size[counted, N[counted]] += 2 * np.abs(g[counted])
    chain = (max(T, W.shape[0]) / 16 + 16 if act == "bf16" else max(T, W.shape[0]) / 2 + 2) * U32
    rel = 2 * off[:, None] + r16 + 8 * U32
    within("dh", dh, DH, r16 * np.abs(DH) + (rel + chain) * (size @ np.abs(W)) + 1e-30)
    Hc = np.where(counted[:, None], H, 0.0)
    within("dw", dw, DW, r16 * np.abs(DW) + ((rel + chain) * size).T @ np.abs(Hc) + 1e-30)
    return loss, lse, dh, dw


SHAPES = [(1, 8, 1), (1, 64, 2), (2, 72, 7), (5, 64, 255), (3, 128, 256), (33, 136, 257), (64, 520, 300),
          (255, 64, 1000), (256, 512, 512), (257, 72, 777), (300, 264, 3001), (700, 128, 5000), (1030, 192, 130)]


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,V", SHAPES)
def test_loss_and_gradients(T, d, V, act):
    print(f"\n[gpu] vocab_loss T={T} d={d} V={V} {act}", flush=True)
    rng = np.random.default_rng([T, d, V])
    h, w = normal(rng, (T, d), act), normal(rng, (V, d), act, 2.0 / np.sqrt(d))
    _check(h, w, _targets(rng, T, V, 0.3 if T > 1 else 0.0), act)


# Sizes that take the widest tiles, forward (V) or backward (d), with fewer and
# fewer counted tokens: the tile goes by their number, which the launch does not
# know.
@pytest.mark.parametrize("ignored", [0.0, 0.3, 0.6, 0.97])
@pytest.mark.parametrize("T,d,V", [(1111, 72, 20021), (1000, 64, 16384), (1500, 2056, 2300), (2500, 2504, 2490)])
def test_wide_tiles_by_the_counted_tokens(T, d, V, ignored):
    print(f"\n[gpu] vocab_loss T={T} d={d} V={V} ignored={ignored}", flush=True)
    rng = np.random.default_rng([T, int(100 * ignored)])
    h, w = normal(rng, (T, d), "bf16"), normal(rng, (V, d), "bf16", 2.0 / np.sqrt(d))
    _check(h, w, _targets(rng, T, V, ignored), "bf16")


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T", [2047, 2049, 16385, 70000])
def test_many_tokens(T, act):
    """Tokens past one round of the gather, in workgroups of 4, 16 and 64 or more."""
    print(f"\n[gpu] vocab_loss T={T} {act}", flush=True)
    rng = np.random.default_rng(T)
    d, V = 72, 40
    h, w = normal(rng, (T, d), act), normal(rng, (V, d), act, 0.2)
    _check(h, w, _targets(rng, T, V, 0.4), act, normal(rng, T, "f32"))


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,V,piece", [(1, 64, 20000, 0), (16, 520, 16391, 0), (70, 72, 30000, 4096),
                                         (130, 264, 9000, 8192), (300, 1032, 12001, 0)])
def test_few_tokens_and_a_long_vocabulary(T, d, V, piece, act):
    """dh's sum over the vocabulary split over workgroups, pieces or not."""
    print(f"\n[gpu] vocab_loss T={T} d={d} V={V} piece={piece} {act}", flush=True)
    rng = np.random.default_rng([T, V])
    h, w = normal(rng, (T, d), act), normal(rng, (V, d), act, 2.0 / np.sqrt(d))
    _check(h, w, _targets(rng, T, V, 0.2 if T > 1 else 0.0), act, piece=piece)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,V,piece", [(9000, 520, 256, 0), (20000, 64, 1, 0), (6000, 264, 700, 256)])
def test_many_tokens_and_a_small_vocabulary(T, d, V, piece, act):
    """dw's sum over the tokens split over workgroups."""
    print(f"\n[gpu] vocab_loss T={T} d={d} V={V} piece={piece} {act}", flush=True)
    rng = np.random.default_rng([T, V])
    h, w = normal(rng, (T, d), act), normal(rng, (V, d), act, 2.0 / np.sqrt(d))
    _check(h, w, _targets(rng, T, V, 0.2), act, piece=piece)


def test_the_largest_tiles():
    T, d, V = 4000, 4096, 4000
    print(f"\n[gpu] vocab_loss T={T} d={d} V={V}", flush=True)
    rng = np.random.default_rng(T)
    h, w = normal(rng, (T, d), "bf16"), normal(rng, (V, d), "bf16", 2.0 / np.sqrt(d))
    _check(h, w, _targets(rng, T, V, 0.05), "bf16")


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("piece", [1, 256, 300, 512, 100000])
def test_pieces(piece, act):
    print(f"\n[gpu] vocab_loss piece={piece} {act}", flush=True)
    rng = np.random.default_rng(piece)
    T, d, V = 310, 200, 1300
    h, w, t = normal(rng, (T, d), act), normal(rng, (V, d), act, 0.1), _targets(rng, T, V, 0.2)
    dloss = normal(rng, T, "f32")
    dloss[::5] = 0
    _check(h, w, t, act, dloss, -0.5, piece)


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_no_token_counted(act):
    rng = np.random.default_rng(2)
    h, w = normal(rng, (40, 64), act), normal(rng, (300, 64), act)
    t = torch.full((40,), -100, dtype=torch.int64, device="cuda")
    loss, lse = model.vocab_loss(h, w, t)
    dh, dw = model.vocab_loss_backward(h, w, t, lse, piece=256)
    torch.cuda.synchronize()
    assert torch.all(loss == 0) and torch.all(lse == 0) and torch.all(dh == 0) and torch.all(dw == 0)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 72])
def test_rows_that_are_not_counted_and_gaps_between_rows_are_never_used(act, d):
    rng = np.random.default_rng(d)
    T, V = 70, 600
    h, w, t = normal(rng, (T, d), act), normal(rng, (V, d), act), _targets(rng, T, V, 0.4)
    want = model.vocab_loss(h, w, t)
    grads = model.vocab_loss_backward(h, w, t, want[1])
    N = t.cpu().numpy()
    bad = torch.from_numpy((N < 0) | (N >= V)).cuda()
    h2 = h.clone()
    h2[bad] = float("nan")
    h2[bad.nonzero()[0]] = float("inf")
    h2, w2 = strided(h2, 8), strided(w, 24, float("inf"))
    got = model.vocab_loss(h2, w2, t)
    grads2 = model.vocab_loss_backward(h2, w2, t, got[1])
    torch.cuda.synchronize()
    for a, b in zip(want + grads, got + grads2):
        assert torch.equal(a, b)


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_large_logits(act):
    """Logits of several hundred: exponentials only of differences."""
    rng = np.random.default_rng(4)
    h, w = normal(rng, (50, 128), act, 8.0), normal(rng, (700, 128), act, 3.0)
    _check(h, w, _targets(rng, 50, 700, 0.1), act)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("T", [20, 9000])
def test_a_gradient_that_is_not_finite_stays_with_its_token(T, bad):
    rng = np.random.default_rng(9)
    h, w, t = normal(rng, (T, 64), "bf16"), normal(rng, (300, 64), "bf16"), _targets(rng, T, 300, 0.0)
    _, lse = model.vocab_loss(h, w, t)
    dloss = normal(rng, T, "f32")
    dloss[7] = 0
    want, _ = model.vocab_loss_backward(h, w, t, lse, dloss)
    dloss[7] = bad
    got, _ = model.vocab_loss_backward(h, w, t, lse, dloss)
    torch.cuda.synchronize()
    keep = [i for i in range(T) if i != 7]
    assert torch.equal(got[keep], want[keep]) and not torch.isfinite(got[7]).any()


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_slices_of_targets_and_gradients(act):
    """Targets as a token sequence shifted by one, loss gradients from the middle of a tensor."""
    rng = np.random.default_rng(10)
    h, w = normal(rng, (33, 72), act), normal(rng, (300, 72), act)
    ids, g = _targets(rng, 34, 300, 0.2), normal(rng, 36, "f32")
    t, dloss = ids[1:], g[3:]
    want = _check(h, w, t.clone(), act, dloss.clone())
    lse = torch.empty(34, device="cuda")[1:]
    lse.copy_(want[1])
    loss2, _ = model.vocab_loss(h, w, t)
    got = model.vocab_loss_backward(h, w, t, lse, dloss)
    torch.cuda.synchronize()
    assert torch.equal(loss2, want[0]) and all(torch.equal(a, b) for a, b in zip(got, want[2:]))


def test_a_row_that_is_not_finite_shows_in_its_loss_only():
    rng = np.random.default_rng(6)
    h, w, t = normal(rng, (20, 64), "bf16"), normal(rng, (300, 64), "bf16"), _targets(rng, 20, 300, 0.0)
    want, _ = model.vocab_loss(h, w, t)
    h[3, 5] = float("nan")
    loss, _ = model.vocab_loss(h, w, t)
    torch.cuda.synchronize()
    assert torch.isnan(loss[3])
    keep = [i for i in range(20) if i != 3]
    assert torch.equal(loss[keep], want[keep])


def test_the_mean_gradient_of_a_broadcast_upstream():
    rng = np.random.default_rng(7)
    h, w, t = normal(rng, (33, 64), "f32"), normal(rng, (90, 64), "f32"), _targets(rng, 33, 90, 0.5)
    n = int(((t >= 0) & (t < 90)).sum())
    _, lse = model.vocab_loss(h, w, t)
    one = torch.full((), 1.0 / n, device="cuda").expand(33)
    a = model.vocab_loss_backward(h, w, t, lse)
    b = model.vocab_loss_backward(h, w, t, lse, one)
    for x, y in zip(a, b):
        assert torch.allclose(x, y, rtol=4 * U32, atol=0)


def test_gradient_against_differences():
    rng = np.random.default_rng(8)
    T, d, V, step = 12, 64, 50, 2.0 ** -7
    h, w, t = normal(rng, (T, d), "f32"), normal(rng, (V, d), "f32", 0.2), _targets(rng, T, V, 0.2)
    dloss = normal(rng, T, "f32")
    _, lse = model.vocab_loss(h, w, t)
    dh, dw = model.vocab_loss_backward(h, w, t, lse, dloss)
    f = lambda a, b: float((model.vocab_loss(a, b, t)[0].double() * dloss.double()).sum())  # noqa: E731
    for k in range(4):
        u, v = normal(rng, (T, d), "f32"), normal(rng, (V, d), "f32")
        got = float((dh.double() * u.double()).sum() + (dw.double() * v.double()).sum())
        diff = (f(h + step * u, w + step * v) - f(h - step * u, w - step * v)) / (2 * step)
        # third derivatives of about (u w + h v)^3 ~ 8^3 a token, times step^2 / 6; the losses' rounding / step
        assert abs(diff - got) < 0.06 + 1e-3 * abs(got), k


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_repeats_to_the_bit_and_on_another_stream(act):
    rng = np.random.default_rng(12)
    h, w, t = normal(rng, (400, 128), act), normal(rng, (2000, 128), act), _targets(rng, 400, 2000, 0.2)
    loss, lse = model.vocab_loss(h, w, t)
    dh, dw = model.vocab_loss_backward(h, w, t, lse, piece=512)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        loss2, lse2 = model.vocab_loss(h, w, t)
        dh2, dw2 = model.vocab_loss_backward(h, w, t, lse2, piece=512)
    s.synchronize()
    torch.cuda.synchronize()
    for a, b in ((loss, loss2), (lse, lse2), (dh, dh2), (dw, dw2)):
        assert torch.equal(a, b)


def test_no_tokens():
    w = torch.ones((100, 64), dtype=torch.bfloat16, device="cuda")
    h, t = w[:0], torch.empty(0, dtype=torch.int64, device="cuda")
    loss, lse = model.vocab_loss(h, w, t)
    dh, dw = model.vocab_loss_backward(h, w, t, lse)
    assert loss.shape == (0,) and dh.shape == (0, 64) and torch.all(dw == 0)


def test_vocabulary_past_two_to_the_31_elements():
    V, d, T = 540000, 4096, 6
    print(f"\n[gpu] vocab_loss T={T} d={d} V={V}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(1)
    h = torch.randn((T, d), generator=g, device="cuda").bfloat16()
    w = torch.empty((V, d), dtype=torch.bfloat16, device="cuda")
    for i in range(0, V, 60000):
        w[i:i + 60000] = torch.randn((60000, d), generator=g, device="cuda").mul_(0.02).bfloat16()
    t = torch.tensor([0, V - 1, 270000, V, V - 2, 5], device="cuda")
    loss, lse = model.vocab_loss(h, w, t)
    dh, dw = model.vocab_loss_backward(h, w, t, lse)
    l = torch.cat([h.float() @ w[i:i + 60000].float().t() for i in range(0, V, 60000)], 1).double()
    counted = torch.tensor([0, 1, 2, 4, 5], device="cuda")
    LSE = torch.logsumexp(l[counted], 1)
    LOSS = LSE - l[counted, t[counted]]
    within("loss", loss[counted], f64(LOSS), 1e-4)
    p = (l[counted] - LSE[:, None]).exp()
    p[torch.arange(5, device="cuda"), t[counted]] -= 1
    p /= 5
    for rows in (slice(0, 8), slice(V - 8, V), slice(269996, 270004)):
        want, size = f64(p[:, rows].t() @ h[counted].double()), f64(p[:, rows].abs().t() @ h[counted].double().abs())
        within("dw", dw[rows], want, U16 * np.abs(want) + 1.2 * U16 * size)
    DH = torch.zeros((5, d), dtype=torch.float64, device="cuda")
    size = torch.zeros_like(DH)
    for i in range(0, V, 60000):
        DH += p[:, i:i + 60000] @ w[i:i + 60000].double()
        size += p[:, i:i + 60000].abs() @ w[i:i + 60000].double().abs()
    within("dh", dh[counted], f64(DH), U16 * np.abs(f64(DH)) + 1.2 * U16 * f64(size))
    assert torch.all(dh[3] == 0) and loss[3] == 0


@pytest.mark.parametrize("bad", ["h", "w", "target", "lse", "dloss", "width", "piece"])
def test_refusals(bad):
    h = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((10, 64), dtype=torch.bfloat16, device="cuda")
    t, f = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(4, device="cuda")
    args = dict(h=h, w=w, target=t, lse=f, dloss=f)
    piece = 0
    if bad == "h":
        args["h"] = h.half()
    elif bad == "w":
        args["w"] = w[:, :56]
    elif bad == "target":
        args["target"] = t.int()
    elif bad == "lse":
        args["lse"] = f[:3]
    elif bad == "dloss":
        args["dloss"] = f.double()
    elif bad == "width":
        args["h"], args["w"] = h[:, :60].contiguous(), w[:, :60].contiguous()
    else:
        piece = -1
    with pytest.raises((ValueError, px.PoetxError)):
        model.vocab_loss_backward(*args.values(), piece=piece)
