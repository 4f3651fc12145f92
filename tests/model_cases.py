"""Shared by the GPU tests of the operators around the layer: seeded inputs,
float64 views and elementwise bounds."""

import numpy as np
import torch

U16 = 2.0 ** -8    # largest relative rounding to bfloat16 (8 significant bits: half a step of 2^-7 at 1)
U32 = 2.0 ** -24   # to float32

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def normal(rng, shape, dtype, scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).to(DTYPES[dtype]).cuda()


def strided(t, pad, fill=float("nan")):
    """The same matrix with `pad` more elements between its rows, all `fill`."""
    full = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device=t.device)
    full[:, :t.shape[1]] = t
    return full[:, :t.shape[1]]


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def within(name, got, want, bound):
    """|got - want| <= bound elementwise (and finite)."""
    got = f64(got) if isinstance(got, torch.Tensor) else got
    off = np.abs(got - want)
    bad = ~(off <= bound)
    assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size} past the bound, worst "
                           f"{np.nanmax(np.where(bad, off / np.maximum(bound, 1e-300), 0)):.3g} times it; first at "
                           f"{np.argwhere(bad)[0].tolist()}")
