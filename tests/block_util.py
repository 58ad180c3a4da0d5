"""Helpers of the gated recurrent block's GPU tests: seeded inputs on the
device and their exact fp64 copies, and the comparison with a stated bound."""
from __future__ import annotations

import numpy as np
import torch

HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}      # finfo.eps / 2


def rand(seed, *shape, dtype=torch.float32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def close(got, want, bound, name=""):
    """|got - want| <= the fp32 evaluation's bound, plus one rounding of the
    result to its type, plus its smallest normal number."""
    g = f64(got)
    assert g.shape == want.shape, (name, g.shape, want.shape)
    assert np.isfinite(g).all(), f"{name}: non-finite values"
    half = HALF_STEP[got.dtype]
    tol = bound * (1.0 + half) + half * np.abs(want) + 2.0 ** -126
    bad = np.abs(g - want) > tol
    if bad.any():
        i = np.unravel_index(np.argmax(np.abs(g - want) / tol), g.shape)
        raise AssertionError(f"{name}: {bad.sum()} of {bad.size} off, worst at {i}: {g[i]} for {want[i]}, allowed {tol[i]}")


def guarded(shape, dtype, pad=512):
    """A tensor of this shape inside a larger buffer filled with a pattern, and
    a check that nothing around it was written."""
    n = int(np.prod(shape))
    buf = torch.full((n + 2 * pad,), 7.0, device="cuda").to(dtype)
    inner = buf[pad:pad + n].view(shape)

    def check():
        assert bool((buf[:pad].float() == 7.0).all()) and bool((buf[pad + n:].float() == 7.0).all()), "written outside"
    return inner, check


def along_its_signs(loss, inputs, name, grad, h, noise):
    """Central differences of loss(inputs) along the signs of its gradient by inputs[name]: returns the difference to
    sum |grad|, where every value counts with its full weight, and what is allowed of it: 1e-4 for the third
    derivative (h = 0.02 leaves up to 5e-5 of the recurrence's, in 64 bits), and 4 times `noise`, the loss's
    rounding in quadrature, for each of the two losses."""
    sign = (grad < 0) * -2.0 + 1.0
    hi, lo = ({**inputs, name: inputs[name] + d * sign} for d in (h, -h))
    want = abs(grad).sum()
    return abs((loss(hi) - loss(lo)) / (2 * h) - want), 1e-4 * want + 4 * 2 ** 0.5 * noise / (2 * h)
