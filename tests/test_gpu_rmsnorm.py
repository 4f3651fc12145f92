"""RMS norm with the residual's addition, its int8 rows and its backward,
against the float64 form.

Bounds: a value computed in float32 from a row of n is off by the error of the
mean (a sum of n squares in a tree of depth ~ n / 2048 + 14 additions, halved
by the square root) and a handful of roundings: under 16 u32 relative for the
widths here. bfloat16 outputs add u16 of the value.
"""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from model_cases import DTYPES, U16, U32, f64, normal, strided, within  # noqa: E402
from oracle import model_oracle as M  # noqa: E402
from orthogonal_equivalence_amd import model  # noqa: E402
from orthogonal_equivalence_amd import model_ops as mo  # noqa: E402
from orthogonal_equivalence_amd import poetx as px  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible AMD GPU"
    torch.cuda.init()


def _out(act):
    return U16 if act == "bf16" else 0.0


# every width class of the kernels and its edges, one token to many
SHAPES = [(1, 8), (3, 16), (5, 504), (2, 512), (7, 520), (1, 1024), (9, 1032), (4, 2048), (3, 2056), (1, 4096),
          (6, 4104), (2, 8192), (3, 8200), (2, 16384), (1, 16392), (2, 32768), (2, 32776), (1, 70000), (1500, 72),
          (1030, 1032), (600, 2064), (7, 64), (9000, 64), (13, 128), (9001, 136), (4500, 256), (6, 264), (700, 6152),
          (513, 8200)]


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,n", SHAPES)
def test_forward_and_backward(T, n, act):
    print(f"\n[gpu] rms_norm T={T} n={n} {act}", flush=True)
    rng = np.random.default_rng([T, n])
    x, r = normal(rng, (T, n), act), normal(rng, (T, n), act, 3.0)
    dy, dh = normal(rng, (T, n), act), normal(rng, (T, n), act)
    gain = normal(rng, n, "f32")
    h, y, rstd = model.rms_norm(x, gain, r, 1e-5)
    dx, dgain = model.rms_norm_backward(dy, h, rstd, gain, dh)
    torch.cuda.synchronize()
    H, Y, R = M.rms_norm(f64(x), f64(gain), f64(r), 1e-5)
    e = 16 * U32
    within("h", h, H, (_out(act) + U32) * np.abs(H))
    within("rstd", rstd, R, e * R)
    within("y", y, Y, (_out(act) + e) * np.abs(Y) + 1e-30)
    hd, rs = f64(h), f64(rstd)[:, None]
    DX, DG = M.rms_norm_backward(f64(dy), hd, f64(gain), dh=f64(dh), rstd=f64(rstd))
    u, dyg = hd * rs, f64(dy) * f64(gain)
    size = rs * (np.abs(dyg) + np.abs(u) * np.mean(np.abs(dyg * u), axis=1, keepdims=True)) + np.abs(f64(dh))
    within("dx", dx, DX, _out(act) * np.abs(DX) + e * size)
    # dgain: at most T / groups additions in a group, then 64 + 4 over the groups
    within("dgain", dgain, DG, (T / mo.poetx_rmsnorm_ws_bytes(T, n) * 4 * n + 72) * U32 * np.sum(np.abs(f64(dy) * u), 0))


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,n", [(1, 16), (5, 512), (3, 1040), (2, 2048), (1, 4096), (33, 5120), (2, 16384), (1, 32784),
                                 (700, 272)])
def test_int8_rows(T, n, act):
    print(f"\n[gpu] rms_norm_q8 T={T} n={n} {act}", flush=True)
    rng = np.random.default_rng([T, n, 1])
    x, r, gain = normal(rng, (T, n), act), normal(rng, (T, n), act), normal(rng, n, "f32")
    h, q, scale = model.rms_norm_q8(x, gain, r)
    q2, scale2 = model.quantize_rows(x)
    torch.cuda.synchronize()
    H, Y, _ = M.rms_norm(f64(x), f64(gain), f64(r))
    within("h", h, H, (_out(act) + U32) * np.abs(H))
    for name, codes, s, v, e in (("norm", q, scale, Y, 20 * U32), ("rows", q2, scale2, f64(x), 4 * U32)):
        _, S = M.quantize_rows(v)
        within(name + " scale", s, S, e * S)
        # a code is the nearest whole number to v / scale, computed with e
        within(name + " codes", codes, v / S[:, None], 0.5 + 127 * e)
        assert int(codes.abs().max()) == 127


def test_no_residual_and_the_stream_itself():
    rng = np.random.default_rng(5)
    x, gain = normal(rng, (9, 640), "bf16"), normal(rng, 640, "f32")
    h, y, rstd = model.rms_norm(x, gain)
    assert h is x
    _, Y, _ = M.rms_norm(f64(x), f64(gain))
    within("y", y, Y, (U16 + 16 * U32) * np.abs(Y))
    dy = normal(rng, (9, 640), "bf16")
    dx, _ = model.rms_norm_backward(dy, x, rstd, gain)
    DX, _ = M.rms_norm_backward(f64(dy), f64(x), f64(gain), rstd=f64(rstd))
    within("dx", dx, DX, U16 * np.abs(DX) + 1e-5)


def test_rstd_of_some_of_the_tokens():
    rng = np.random.default_rng(12)
    x, gain, dy = normal(rng, (9, 640), "bf16"), normal(rng, 640, "f32"), normal(rng, (9, 640), "bf16")
    _, _, rstd = model.rms_norm(x, gain)
    got = model.rms_norm_backward(dy[3:], x[3:], rstd[3:], gain)
    want = model.rms_norm_backward(dy[3:].clone(), x[3:].clone(), rstd[3:].clone(), gain)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_strided_stream_without_a_residual():
    rng = np.random.default_rng(8)
    x, gain, dy = strided(normal(rng, (9, 640), "bf16"), 8), normal(rng, 640, "f32"), normal(rng, (9, 640), "bf16")
    h, y, rstd = model.rms_norm(x, gain)
    assert h is x
    got = model.rms_norm_backward(dy, h, rstd, gain)
    want = model.rms_norm_backward(dy, x.contiguous(), rstd, gain)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("n", [256, 4096, 40000])
def test_in_place_and_strided(n):
    print(f"\n[gpu] rms_norm in place, strided n={n}", flush=True)
    rng = np.random.default_rng(n)
    x, r, gain = normal(rng, (5, n), "bf16"), normal(rng, (5, n), "bf16"), normal(rng, n, "f32")
    dy, dh = normal(rng, (5, n), "bf16"), normal(rng, (5, n), "bf16")
    h, y, rstd = model.rms_norm(x, gain, r)
    hs, ys, rs = model.rms_norm(strided(x, 8), gain, strided(r, 24))
    assert torch.equal(h, hs) and torch.equal(y, ys) and torch.equal(rstd, rs)
    dx, dg = model.rms_norm_backward(dy, h, rstd, gain, dh)
    dxs, dgs = model.rms_norm_backward(strided(dy, 16), h, rstd, gain, strided(dh, 8))
    assert torch.equal(dx, dxs) and torch.equal(dg, dgs)
    # h over the residual, dx over dh
    r2, y2, dh2 = r.clone(), torch.empty_like(y), dh.clone()
    mo.poetx_rmsnorm_forward(5, n, px.POETX_BF16, x, n, r2, n, gain, 1e-6, r2, y2, None)
    mo.poetx_rmsnorm_backward(5, n, px.POETX_BF16, dy, n, r2, rstd, gain, dh2, n, dh2, None)
    torch.cuda.synchronize()
    assert torch.equal(r2, h) and torch.equal(y2, y) and torch.equal(dh2, dx)


def test_zero_rows_and_values_that_are_not_finite():
    n = 1024
    x = torch.zeros((6, n), dtype=torch.bfloat16, device="cuda")
    x[1, 3] = float("nan")
    x[2, 5] = float("inf")
    x[3, 7] = 2.0 ** -120
    x[4] = 1.0
    x[5] = -3e38
    gain = torch.ones(n, device="cuda")
    _, y, _ = model.rms_norm(x, gain)
    _, q, scale = model.rms_norm_q8(x, gain)
    rq, rscale = model.quantize_rows(x)
    torch.cuda.synchronize()
    assert torch.all(y[0] == 0) and torch.all(q[0] == 0) and scale[0] == 1
    assert torch.isnan(y[1]).all() and torch.isnan(scale[1])
    assert torch.isnan(y[2, 5]) and not torch.isfinite(scale[2])
    assert torch.all(y[4] == 1) and torch.all(q[4] == 127)
    assert torch.all(y[5] == 0)   # the square overflows float32: rstd 0, as the formula gives
    assert torch.isnan(rscale[1]) and torch.isinf(rscale[2]) and rscale[3] == 1 and torch.all(rq[3] == 0)


def test_no_tokens():
    gain = torch.ones(64, device="cuda")
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    h, y, rstd = model.rms_norm(e, gain, e)
    dx, dgain = model.rms_norm_backward(e, h, rstd, gain, e)
    assert y.shape == (0, 64) and dx.shape == (0, 64) and torch.all(dgain == 0)
    assert model.rms_norm_q8(e, gain)[1].shape == (0, 64)


def test_gradient_against_differences():
    rng = np.random.default_rng(9)
    T, n, eps = 3, 264, 1e-3
    x, r, gain = normal(rng, (T, n), "f32"), normal(rng, (T, n), "f32"), normal(rng, n, "f32")
    dy = normal(rng, (T, n), "f32")
    h, _, rstd = model.rms_norm(x, gain, r, eps)
    dx, dgain = model.rms_norm_backward(dy, h, rstd, gain)
    step = 2.0 ** -8
    for k in range(6):
        v = normal(rng, (T, n), "f32")
        f = lambda s: float((dy.double() * model.rms_norm(x + s * v, gain, r, eps)[1].double()).sum())  # noqa: E731
        got = float((dx.double() * v.double()).sum())
        # truncation step^2 times third derivatives of order 1 a term, rounding u32 |y dy| / step
        assert abs((f(step) - f(-step)) / (2 * step) - got) < 5e-2, k


def test_broadcast_gradient_is_copied_out():
    rng = np.random.default_rng(10)
    x, gain = normal(rng, (4, 128), "f32"), normal(rng, 128, "f32")
    h, _, rstd = model.rms_norm(x, gain)
    one = torch.ones((), device="cuda").expand(4, 128)
    dx, dg = model.rms_norm_backward(one, h, rstd, gain, one)
    dx2, dg2 = model.rms_norm_backward(one.contiguous(), h, rstd, gain, one.contiguous())
    assert torch.equal(dx, dx2) and torch.equal(dg, dg2)


def test_repeats_to_the_bit_and_on_another_stream():
    rng = np.random.default_rng(11)
    x, dy, gain = normal(rng, (3000, 1536), "bf16"), normal(rng, (3000, 1536), "bf16"), normal(rng, 1536, "f32")
    torch.cuda.synchronize()
    h, y, rstd = model.rms_norm(x, gain)
    dx, dg = model.rms_norm_backward(dy, h, rstd, gain)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _, y2, rstd2 = model.rms_norm(x, gain)
        dx2, dg2 = model.rms_norm_backward(dy, x, rstd2, gain)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(dx, dx2) and torch.equal(dg, dg2)


def test_rows_past_two_to_the_31_elements():
    T, n = 300000, 8192
    print(f"\n[gpu] rms_norm T={T} n={n}", flush=True)
    x = torch.ones((T, n), dtype=torch.bfloat16, device="cuda")
    x[-1] = torch.arange(n, device="cuda").remainder(7).to(torch.bfloat16)
    gain = torch.ones(n, device="cuda")
    _, y, rstd = model.rms_norm(x, gain)
    _, Y, _ = M.rms_norm(f64(x[-2:]), f64(gain))
    within("y", y[-2:], Y, (U16 + 16 * U32) * np.abs(Y))
    dx, dgain = model.rms_norm_backward(x, x, rstd, gain, x)
    DX, _ = M.rms_norm_backward(f64(x[-2:]), f64(x[-2:]), f64(gain), dh=f64(x[-2:]), rstd=f64(rstd[-2:]))
    within("dx", dx[-2:], DX, U16 * np.abs(DX) + 1e-4)
    want = (T - 1) + f64(x[-1]) ** 2 * f64(rstd[-1:])
    within("dgain", dgain, want, 1e-4 * want)


def test_more_rows_than_one_grid_dimension_holds():
    T, n = (1 << 24) + 5, 1040   # 2^24 workgroups of 256 threads are 2^32 threads
    print(f"\n[gpu] quantize_rows T={T} n={n}", flush=True)
    x = torch.zeros((T, n), dtype=torch.bfloat16, device="cuda")
    for i in (0, (1 << 21) - 1, 1 << 21, 1 << 24, T - 1):
        x[i, i % n] = 1 + i % 7
    q, scale = model.quantize_rows(x)
    torch.cuda.synchronize()
    for i in (0, (1 << 21) - 1, 1 << 21, 1 << 24, T - 1):
        assert int(q[i, i % n]) == 127 and int(q[i].abs().sum()) == 127
        assert float(scale[i]) == pytest.approx((1 + i % 7) / 127, rel=1e-6)
    assert int((scale != 1).sum()) == 5


@pytest.mark.parametrize("bad", ["shape", "dtype", "columns", "host", "gain", "int"])
def test_refusals(bad):
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    gain, res = torch.ones(64, device="cuda"), x
    if bad == "shape":
        res = x[:2]
    elif bad == "dtype":
        res = x.float()
    elif bad == "columns":
        x = torch.zeros((64, 4), dtype=torch.bfloat16, device="cuda").t()
        res = x
    elif bad == "host":
        x = res = x.cpu()
    elif bad == "gain":
        gain = gain.bfloat16()
    else:
        x = res = x.to(torch.int8)
    with pytest.raises(ValueError):
        model.rms_norm(x, gain, res)
    with pytest.raises(px.PoetxError):  # 60 features
        model.rms_norm(torch.zeros((4, 60), dtype=torch.bfloat16, device="cuda"), torch.ones(60, device="cuda"))
    with pytest.raises(px.PoetxError):  # rows that do not start on 16 bytes
        z = torch.zeros((4, 68), dtype=torch.bfloat16, device="cuda")
        model.rms_norm(z[:, :64], torch.ones(64, device="cuda"))
