"""The operators around the layer while torch records gradients: they record no
graph, and refuse inputs that would expect one."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from orthogonal_equivalence_amd import model  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible AMD GPU"
    torch.cuda.init()


def _f(*shape):
    return torch.ones(shape, device="cuda")


CALLS = {
    "rms_norm": (model.rms_norm, dict(x=(4, 64), gain=(64,), residual=(4, 64))),
    "rms_norm_q8": (model.rms_norm_q8, dict(x=(4, 64), gain=(64,), residual=(4, 64))),
    "quantize_rows": (model.quantize_rows, dict(x=(4, 64))),
    "rms_norm_backward": (model.rms_norm_backward, dict(dy=(4, 64), h=(4, 64), rstd=(4,), gain=(64,), dh=(4, 64))),
    "linear_i8": (model.linear_i8, dict(xq=(4, 64), x_scale=(4,), wt=(32, 64), w_scale=(32,))),
    "vocab_loss": (model.vocab_loss, dict(h=(4, 64), w=(10, 64), target=(4,))),
    "vocab_loss_backward": (model.vocab_loss_backward, dict(h=(4, 64), w=(10, 64), target=(4,), lse=(4,), dloss=(4,))),
}
INT = dict(xq=torch.int8, wt=torch.int8, target=torch.int64)


def _args(shapes):
    return {k: _f(*s).to(INT.get(k, torch.float32)) for k, s in shapes.items()}


@pytest.mark.parametrize("name,arg", [(n, a) for n, (_, shapes) in CALLS.items() for a in shapes if a not in INT])
def test_an_input_that_requires_a_gradient(name, arg):
    f, shapes = CALLS[name]
    args = _args(shapes)
    want = f(**args)
    args[arg].requires_grad_(True)
    with pytest.raises(ValueError, match="requires a gradient"):
        f(**args)
    with torch.no_grad():
        got = f(**args)
    torch.cuda.synchronize()
    want, got = (x if isinstance(x, tuple) else (x,) for x in (want, got))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_within_an_autograd_function():
    class Loss(torch.autograd.Function):
        @staticmethod
        def forward(ctx, h, w, target):
            loss, lse = model.vocab_loss(h, w, target)
            ctx.save_for_backward(h, w, target, lse)
            return loss

        @staticmethod
        def backward(ctx, g):
            h, w, target, lse = ctx.saved_tensors
            return (*model.vocab_loss_backward(h, w, target, lse, g), None)

    gen = torch.Generator(device="cuda").manual_seed(1)
    h, w = (torch.randn(s, generator=gen, device="cuda").requires_grad_(True) for s in ((12, 64), (40, 64)))
    t = torch.arange(12, device="cuda")
    Loss.apply(h, w, t).sum().backward()
    with torch.no_grad():
        _, lse = model.vocab_loss(h, w, t)
        dh, dw = model.vocab_loss_backward(h, w, t, lse, torch.ones(12, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(h.grad, dh) and torch.equal(w.grad, dw)
