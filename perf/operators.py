"""The operators that surround a POET-X layer in a language model, as timed
cases: the RMS norm of the residual stream (with its backward, or with int8
rows out), the int8 product that serves a merged quantised layer, and the
vocabulary cross entropy with its gradient.

``run`` computes a case with elementary torch operations in float32, or, with
``own`` set, through this package's operators.
"""

import torch

own = False

_DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-6


def listed():
    return [
        # one token of a decoding loop at the 8B width: launch latency
        dict(name="norm_decode", kind="norm", T=1, n=4096, act="bf16"),
        # a training micro-batch of 4 x 2048 tokens at the 8B width
        dict(name="norm_8b", kind="norm", T=8192, n=4096, act="bf16"),
        # forward and backward at the 13B width
        dict(name="norm_train_13b", kind="norm_train", T=4096, n=5120, act="bf16"),
        # a float32 model of an odd width, an odd number of tokens
        dict(name="norm_train_f32", kind="norm_train", T=1023, n=1032, act="f32"),
        # one token through norm and MLP-up of a merged int8 layer
        dict(name="serve_one_token", kind="norm_linear", T=1, m=4096, n=14336),
        # 48 sequences decoding together, the 13B down projection
        dict(name="serve_batch", kind="norm_linear", T=48, m=13824, n=5120),
        # a prompt of 777 tokens through a layer of odd widths
        dict(name="linear_prompt", kind="linear", T=777, m=2064, n=5136),
        # a full prefill batch, the 8B MLP-up
        dict(name="linear_prefill", kind="linear", T=8192, m=4096, n=14336),
        # the float32 test model with a small vocabulary
        dict(name="loss_train_f32", kind="loss_train", T=256, d=512, V=1000, act="f32", ignored=0.25),
        # evaluation: loss only, odd sizes throughout
        dict(name="loss_eval", kind="loss", T=1111, d=2056, V=50021, act="bf16", ignored=0.5),
        # a training micro-batch at the 8B width
        dict(name="loss_train", kind="loss_train", T=4096, d=4096, V=32768, act="bf16", ignored=0.1),
        # the largest: 4 x 2048 tokens and a large vocabulary
        dict(name="loss_train_large", kind="loss_train", T=8192, d=4096, V=131072, act="bf16", ignored=0.0),
    ]


def _log_int(rng, lo, hi, step=1):
    """Log-uniform multiple of step in [lo, hi]."""
    v = lo * (hi / lo) ** rng.random()
    return max(lo, int(v) // step * step)


def draw(rng):
    kind = rng.choice(["norm", "norm_train", "norm_linear", "linear", "loss", "loss_train"])
    if kind in ("norm", "norm_train"):
        act = rng.choice(["bf16", "bf16", "f32"])
        n = _log_int(rng, 64, 16384, 8)
        T = _log_int(rng, 1, max(2, min(16384, (1 << 26) // n)))
        return dict(kind=kind, T=T, n=n, act=act)
    if kind in ("norm_linear", "linear"):
        m = _log_int(rng, 128, 14336, 16)
        n = _log_int(rng, 128, 14336, 16)
        T = _log_int(rng, 1, 256 if kind == "norm_linear" else 8192)
        return dict(kind=kind, T=T, m=m, n=n)
    act = rng.choice(["bf16", "bf16", "bf16", "f32"])
    top = 1 if act == "bf16" else 4
    d = _log_int(rng, 64, 4096 // top, 8)
    V = _log_int(rng, 200, 131072 // (2 * top))
    T = _log_int(rng, 1, 8192 // top)
    return dict(kind=kind, T=T, d=d, V=V, act=act, ignored=rng.choice([0.0, 0.1, 0.5, 0.9]))


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _stream_rows(g, T, n, dtype):
    """Rows of a residual stream: N(0, 1) with one feature in 64 eight times
    as large, as such streams have."""
    x = torch.randn((T, n), generator=g, device="cuda")
    return x.mul_(torch.where(torch.rand(n, generator=g, device="cuda") < 1 / 64, 8.0, 1.0)).to(dtype)


def _int8_weight(g, m, n):
    """An int8 weight as a quantised layer exports it, laid out by outputs
    [n][m], and the scale of each output (absmax / 127)."""
    w = torch.randn((n, m), generator=g, device="cuda").mul_(0.02)
    scale = w.abs().amax(1) / 127
    return torch.round(w / scale[:, None]).clamp_(-127, 127).to(torch.int8), scale


def prepare(case, seed):
    g, kind, T = _gen(seed), case["kind"], case["T"]
    s = dict(case=case)
    if kind in ("norm", "norm_train", "norm_linear"):
        dt = _DTYPE[case.get("act", "bf16")]
        n = case["n"] if kind != "norm_linear" else case["m"]
        s["x"] = _stream_rows(g, T, n, dt)
        s["res"] = _stream_rows(g, T, n, dt)
        s["gain"] = 1 + 0.1 * torch.randn(n, generator=g, device="cuda")
        if kind == "norm_train":
            s["dy"] = torch.randn((T, n), generator=g, device="cuda").to(dt)
            s["dh"] = torch.randn((T, n), generator=g, device="cuda").to(dt)
    if kind in ("norm_linear", "linear"):
        s["wt"], s["ws"] = _int8_weight(g, case["m"], case["n"])
    if kind == "linear":
        y = torch.randn((T, case["m"]), generator=g, device="cuda")
        s["xs"] = y.abs().amax(1) / 127
        s["xq"] = torch.round(y / s["xs"][:, None]).clamp_(-127, 127).to(torch.int8)
    if kind in ("loss", "loss_train"):
        dt, d, V = _DTYPE[case["act"]], case["d"], case["V"]
        s["h"] = torch.randn((T, d), generator=g, device="cuda").to(dt)
        s["w"] = torch.randn((V, d), generator=g, device="cuda").mul_(0.02).to(dt)
        # frequent tokens first, as in a tokenizer's vocabulary
        t = (V ** torch.rand(T, generator=g, device="cuda", dtype=torch.float64) - 1).to(torch.int64).clamp_(0, V - 1)
        ignored = torch.rand(T, generator=g, device="cuda") < case["ignored"]
        ignored[0] = False
        s["target"] = torch.where(ignored, -100, t)
    return s


def _plain_norm(s):
    x = s["x"].float() + s["res"].float()
    rstd = torch.rsqrt((x * x).mean(1, keepdim=True) + _EPS)
    return x, rstd, x * rstd * s["gain"]


def _plain(s):
    case = s["case"]
    kind = case["kind"]
    if kind in ("norm", "norm_train"):
        dt = s["x"].dtype
        x, rstd, y = _plain_norm(s)
        out = dict(h=x.to(dt), y=y.to(dt))
        if kind == "norm_train":
            dy = s["dy"].float()
            u = out["h"].float() * rstd
            dyg = dy * s["gain"]
            dx = rstd * (dyg - u * (dyg * u).mean(1, keepdim=True)) + s["dh"].float()
            out.update(dx=dx.to(dt), dgain=(dy * u).sum(0))
        return out
    if kind in ("norm_linear", "linear"):
        out = {}
        if kind == "norm_linear":
            x, _, y = _plain_norm(s)
            out["h"] = x.to(s["x"].dtype)
            amax = y.abs().amax(1)
            xs = torch.where(amax > 0, amax / 127, 1.0)
            xq = torch.round(y / xs[:, None])
        else:
            xs, xq = s["xs"], s["xq"].float()
        z = (xq @ s["wt"].float().t()) * xs[:, None] * s["ws"]
        out["z"] = z.to(torch.bfloat16)
        return out
    dt = s["h"].dtype
    h, w, t = s["h"].float(), s["w"].float(), s["target"]
    valid = (t >= 0) & (t < w.shape[0])
    at = torch.where(valid, t, 0)[:, None]
    logits = h @ w.t()
    top = logits.amax(1, keepdim=True)
    p = torch.exp(logits - top)
    total = p.sum(1, keepdim=True)
    loss = torch.where(valid, (top + torch.log(total) - logits.gather(1, at))[:, 0], 0.0)
    if kind == "loss":
        return dict(loss=loss)
    p = p / total
    p.scatter_add_(1, at, torch.full_like(top, -1.0))
    p *= torch.where(valid, 1.0 / valid.sum().clamp(min=1), 0.0)[:, None]
    return dict(loss=loss, dh=(p @ w).to(dt), dw=(p.t() @ h).to(dt))


def _own(s):
    from orthogonal_equivalence_amd import model

    kind = s["case"]["kind"]
    if kind == "norm":
        h, y, _ = model.rms_norm(s["x"], s["gain"], residual=s["res"], eps=_EPS)
        return dict(h=h, y=y)
    if kind == "norm_train":
        h, y, rstd = model.rms_norm(s["x"], s["gain"], residual=s["res"], eps=_EPS)
        dx, dgain = model.rms_norm_backward(s["dy"], h, rstd, s["gain"], dh=s["dh"])
        return dict(h=h, y=y, dx=dx, dgain=dgain)
    if kind == "norm_linear":
        h, xq, xs = model.rms_norm_q8(s["x"], s["gain"], residual=s["res"], eps=_EPS)
        return dict(h=h, z=model.linear_i8(xq, xs, s["wt"], s["ws"]))
    if kind == "linear":
        return dict(z=model.linear_i8(s["xq"], s["xs"], s["wt"], s["ws"]))
    loss, lse = model.vocab_loss(s["h"], s["w"], s["target"])
    if kind == "loss":
        return dict(loss=loss)
    dh, dw = model.vocab_loss_backward(s["h"], s["w"], s["target"], lse)
    return dict(loss=loss, dh=dh, dw=dw)


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    kind, T = case["kind"], case["T"]
    if kind in ("norm", "norm_train"):
        n, es = case["n"], 2 if case["act"] == "bf16" else 4
        # x, residual -> h, y; the backward adds dy, dh -> dx, dgain
        train = kind == "norm_train"
        return {"bytes": T * n * es * (7 if train else 4) + n * (8 if train else 4), "flops": T * n * (17 if train else 5)}
    if kind in ("norm_linear", "linear"):
        m, n = case["m"], case["n"]
        norm = kind == "norm_linear"
        # the codes between norm and product need not leave the chip
        return {"bytes": m * n + 4 * n + T * n * 2 + (T * m * 6 + 4 * m if norm else T * m + 4 * T),
                "flops": 2 * T * m * n}
    d, V, es = case["d"], case["V"], 2 if case["act"] == "bf16" else 4
    counted = T * (1 - case["ignored"])
    train = kind == "loss_train"
    return {"bytes": es * (counted * d + V * d + (T * d + V * d if train else 0)) + 12 * T,
            "flops": counted * d * V * (6 if train else 2)}


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    f64 = torch.float64
    if kind in ("norm", "norm_train", "norm_linear"):
        a = s["x"].to(f64).add(s["res"].to(f64))
        inv = (a.square().sum(1) / a.shape[1] + _EPS).pow(-0.5).unsqueeze(1)
        unit = a.mul(inv)
        gain = s["gain"].to(f64)
        if kind == "norm":
            return dict(h=a, y=unit.mul(gain))
        if kind == "norm_train":
            # the gradient at the stored stream (in the activation type) with
            # the forward's statistics
            unit_h = a.to(s["x"].dtype).to(f64).mul(inv)
            dy = s["dy"].to(f64)
            inner = torch.einsum("tn,n,tn->t", dy, gain, unit_h).div(a.shape[1]).unsqueeze(1)
            dx = dy.mul(gain).sub(unit_h.mul(inner)).mul(inv).add(s["dh"].to(f64))
            return dict(h=a, y=unit.mul(gain), dx=dx, dgain=torch.einsum("tn,tn->n", dy, unit_h))
        y = unit.mul(gain)
        step = y.abs().max(1).values.div(127).unsqueeze(1)
        rows = y.div(step).round().mul(step)
        return dict(h=a, z=rows @ s["wt"].to(f64).mul(s["ws"].to(f64).unsqueeze(1)).t())
    if kind == "linear":
        rows = s["xq"].to(f64).mul(s["xs"].to(f64).unsqueeze(1))
        return dict(z=rows @ s["wt"].to(f64).mul(s["ws"].to(f64).unsqueeze(1)).t())
    h, w, t = s["h"].to(f64), s["w"].to(f64), s["target"]
    T, V = h.shape[0], w.shape[0]
    counted = torch.nonzero((t >= 0) & (t < V))[:, 0]
    hc, tc = h[counted], t[counted]
    scores = hc @ w.t()
    log_p = scores.sub_(torch.logsumexp(scores, 1, keepdim=True))
    loss = torch.zeros(T, dtype=f64, device=h.device)
    loss[counted] = -log_p[torch.arange(len(tc), device=h.device), tc]
    if kind == "loss":
        return dict(loss=loss)
    grad = log_p.exp_()
    grad[torch.arange(len(tc), device=h.device), tc] -= 1
    grad /= max(1, len(tc))
    dh = torch.zeros_like(h)
    dh[counted] = grad @ w
    return dict(loss=loss, dh=dh, dw=grad.t() @ hc)
