"""The int8 product with scales per token and output against whole-number
sums in float64.

Bounds: the sum is exact; its conversion to float32, two scale products and
(bfloat16) the output's rounding are the only errors: 4 u32 and u16 relative.
"""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from model_cases import DTYPES, U16, U32, f64, within  # noqa: E402
from oracle import model_oracle as M  # noqa: E402
from orthogonal_equivalence_amd import model, synth  # noqa: E402
from orthogonal_equivalence_amd.device import DeviceLayer  # noqa: E402
from orthogonal_equivalence_amd import poetx as px  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible AMD GPU"
    torch.cuda.init()


def _case(T, m, n, seed=0, full=False):
    rng = np.random.default_rng([T, m, n, seed])
    lo, hi = (-128, 128) if full else (-127, 128)
    c = lambda *s: torch.from_numpy(rng.integers(lo, hi, s).astype(np.int8)).cuda()  # noqa: E731
    s = lambda k: torch.from_numpy(rng.uniform(1e-3, 2e-2, k).astype(np.float32)).cuda()  # noqa: E731
    return c(T, m), s(T), c(n, m), s(n)


SHAPES = [(1, 16, 16), (1, 128, 256), (1, 4096, 1024), (2, 144, 272), (3, 2064, 48), (7, 1040, 784), (16, 512, 512),
          (17, 528, 528), (31, 256, 4096), (32, 4096, 2048), (33, 160, 1008), (48, 5120, 640), (64, 1024, 1024),
          (65, 1040, 1040), (127, 272, 16), (128, 2048, 512), (129, 2064, 528), (200, 16, 3000 // 16 * 16),
          (255, 4096, 272), (256, 256, 256), (257, 272, 272), (300, 1024, 2048), (520, 5136, 1552), (777, 640, 784),
          (1030, 1040, 2064), (2050, 128, 5136), (4100, 256, 512)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("T,m,n", SHAPES)
def test_product(T, m, n, out):
    print(f"\n[gpu] linear_i8 T={T} m={m} n={n} {out}", flush=True)
    xq, xs, wt, ws = _case(T, m, n)
    z = model.linear_i8(xq, xs, wt, ws, DTYPES[out])
    torch.cuda.synchronize()
    Z = M.linear_i8(*(a.cpu().numpy() for a in (xq, xs, wt, ws)))
    within("z", z, Z, ((U16 if out == "bf16" else 0.0) + 4 * U32) * np.abs(Z))


@pytest.mark.parametrize("T", [1, 20, 130, 700])
def test_extreme_codes_at_the_widest_sums(T):
    m, n = 131056, 32
    print(f"\n[gpu] linear_i8 T={T} m={m} n={n}, all codes -128", flush=True)
    xq = torch.full((T, m), -128, dtype=torch.int8, device="cuda")
    wt = torch.full((n, m), -128, dtype=torch.int8, device="cuda")
    wt[1::2] = 127
    one = torch.ones(max(T, n), device="cuda")
    z = model.linear_i8(xq, one[:T].clone(), wt, one[:n].clone(), torch.float32)
    want = np.tile(np.where(np.arange(n) % 2, -128.0 * 127 * m, 128.0 * 128 * m), (T, 1))
    within("z", z, want, U32 * np.abs(want))


@pytest.mark.parametrize("T", [1, 24, 100, 600])
def test_output_rows_of_any_stride_and_nothing_else_touched(T):
    print(f"\n[gpu] linear_i8 strided out T={T}", flush=True)
    xq, xs, wt, ws = _case(T, 272, 304, 3, full=True)
    whole = torch.full((T + 2, 304 + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    z = model.linear_i8(xq, xs, wt, ws, out=whole[1:-1, 8:312])
    ref = model.linear_i8(xq, xs, wt, ws)
    torch.cuda.synchronize()
    assert torch.equal(z, ref)
    assert torch.all(whole[0] == 7) and torch.all(whole[-1] == 7)
    assert torch.all(whole[:, :8] == 7) and torch.all(whole[:, 312:] == 7)


def test_scales_that_are_not_finite_stay_in_their_row_or_column():
    xq, xs, wt, ws = _case(5, 64, 64)
    xs[2] = float("nan")
    ws[7] = float("inf")
    z = model.linear_i8(xq, xs, wt, ws, torch.float32)
    torch.cuda.synchronize()
    rows = [0, 1, 3, 4]
    cols = [c for c in range(64) if c != 7]
    assert torch.isnan(z[2]).all() and not torch.isfinite(z[:, 7]).any()
    assert torch.isfinite(z[rows][:, cols]).all()


@pytest.mark.parametrize("T", [1, 5, 100])
def test_some_of_the_tokens_and_outputs(T):
    xq, xs, wt, ws = _case(T + 7, 272, 528)
    z = model.linear_i8(xq, xs, wt, ws)
    part = model.linear_i8(xq[7:], xs[7:], wt[16:], ws[16:])
    torch.cuda.synchronize()
    assert torch.equal(part, z[7:, 16:])


def test_no_tokens():
    xq, xs, wt, ws = _case(1, 64, 64)
    assert model.linear_i8(xq[:0], xs[:0], wt, ws).shape == (0, 64)


@pytest.mark.parametrize("T", [1, 40, 300])
def test_repeats_to_the_bit_and_on_another_stream(T):
    xq, xs, wt, ws = _case(T, 4096, 1040)
    a = model.linear_i8(xq, xs, wt, ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = model.linear_i8(xq, xs, wt, ws)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_rows_past_two_to_the_31_elements():
    T, m, n = 160000, 16, 16384
    print(f"\n[gpu] linear_i8 T={T} m={m} n={n}", flush=True)
    xq, xs, wt, ws = _case(4, m, n)
    x = xq.repeat(T // 4, 1)
    z = model.linear_i8(x, xs.repeat(T // 4), wt, ws)
    torch.cuda.synchronize()
    Z = M.linear_i8(*(a.cpu().numpy() for a in (xq, xs, wt, ws)))
    within("z", z[-4:], Z, (U16 + 4 * U32) * np.abs(Z))


def test_serves_the_exported_weight_of_a_quantised_layer():
    """Norm to int8 rows, then the product of the merged layer's exported
    weight, against the layer's own forward (q = 0) on the same norm."""
    cfg = synth.LayerConfig("serve_xq", 61, 40, 512, 768, 256, 256, "bf16", "i8")
    L = synth.make_layer(cfg, 0)
    layer = DeviceLayer(cfg.m, cfg.n, cfg.b_r, cfg.b_p, cfg.act, cfg.weight, cfg.T)
    layer.load(L)
    layer.cnp_build()
    layer.merge_cycle(1, 0, 1)
    layer.cnp_build()
    w0, scale = layer.export_w0()
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((cfg.T, cfg.m)).astype(np.float32)).bfloat16().cuda()
    gain = torch.ones(cfg.m, device="cuda")
    _, y, _ = model.rms_norm(x, gain)
    want = layer.forward(y)
    _, q, xs = model.rms_norm_q8(x, gain)
    z = model.linear_i8(q, xs, model.linear_i8_weight(w0), scale)
    torch.cuda.synchronize()
    a, b = f64(z), f64(want)
    # the rows' codes are uniform in a step of max / 127 (about 3.2 / 127 of
    # the norm's unit rows): step / sqrt(12) relative, 0.8 %; 2 u16 besides
    assert np.linalg.norm(a - b) / np.linalg.norm(b) < 0.015
    Wd = w0.cpu().numpy().astype(np.float64) * scale.cpu().numpy()
    rows = f64(q) * f64(xs)[:, None]
    within("z", z, rows @ Wd, (U16 + 4 * U32) * np.abs(rows @ Wd) + 1e-6)


@pytest.mark.parametrize("bad", ["xq", "x_scale", "wt", "w_scale", "out", "width"])
def test_refusals(bad):
    xq, xs, wt, ws = _case(4, 64, 64)
    out = torch.empty((4, 64), dtype=torch.bfloat16, device="cuda")
    if bad == "xq":
        xq = xq.float()
    elif bad == "x_scale":
        xs = xs[:3]
    elif bad == "wt":
        wt = wt[:, :48]
    elif bad == "w_scale":
        ws = ws.double()
    elif bad == "out":
        out = out.half()
    else:
        with pytest.raises(px.PoetxError):
            model.linear_i8(xq[:, :56].contiguous(), xs, wt[:, :56].contiguous(), ws)
        return
    with pytest.raises(ValueError):
        model.linear_i8(xq, xs, wt, ws, out=out)
