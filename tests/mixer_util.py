"""Comparison of the chunked delta rule with its step-by-step definition.

A chunk of 64 steps passes through five products one after the other (K S, T X,
P U, Q S, K^T U).  In each, a computed operand is off by at most EPS relative:
bf16 io carries it in two bf16 terms, whose second is rounded by 2^-18 of the
value, and drops the product of the second terms, 2^-18 again (the first
exponentials' and sums' fp32 errors are below that): 2^-17.  fp32 io rounds
products and sums of up to 128 terms, in quadrature 2^-24 * sqrt(128) < 2^-20.
Errors of different products are independent; a state carries them on without
making them larger where |k| <= 1 and beta <= 2, so n chunks and five products add
in quadrature.  A product's operands cancel at most by the two terms of
X = V - K S, which are as large as the values themselves: a factor of 2.  So the
error's root mean square over a tensor is at most

    t = EPS * 2 * sqrt(5 n)

of the values' (or, for dg and dbeta, of the sums' terms), and a single element,
of some million normal ones, is off by less than 8 of that, taken twice for
heads that are unlike: 16 t."""
import numpy as np

import block_util as U
import torch

EPS = {torch.float32: 2.0 ** -20, torch.bfloat16: 2.0 ** -17}


def close(got, want, io, steps, name, size=None, half=None):
    """got against want: io the inputs' type, size the root mean square that the error is measured by (want's), half the
    rounding of the outputs' type (got's)."""
    g = U.f64(got)
    assert g.shape == want.shape, (name, g.shape, want.shape)
    if g.size == 0:
        return
    assert np.isfinite(g).all(), f"{name}: not finite"
    half = U.HALF_STEP[got.dtype] if half is None else half
    rms = max(float(np.sqrt(np.mean(want * want))), 0.0 if size is None else size)
    t = EPS[io] * 2.0 * np.sqrt(5.0 * max(1, -(-steps // 64))) * rms + 2.0 ** -126
    d = np.abs(g - want) - half * np.abs(want)
    worst, whole = float(d.max()), float(np.sqrt(np.mean(np.maximum(d, 0.0) ** 2)))
    assert worst <= 16.0 * t and whole <= t, f"{name}: worst {worst / t:.2f} t, rms {whole / t:.2f} t ({rms:.3g} rms)"


def rms(a):
    return float(np.sqrt(np.mean(np.square(a)))) if np.size(a) else 0.0


def delta_inputs(B, T, Hk, H, K, V, dtype, state=True, packed=False, seed=0, n=None):
    """Unit keys, memories of 2 to some hundred steps, beta in (0, 1); packed: q, k, v as column ranges of one tensor."""
    q, k = (U.rand(seed + i, B, T, Hk, K) for i in range(2))
    q, k = (t / t.norm(dim=-1, keepdim=True) for t in (q, k))
    v = U.rand(seed + 2, B, T, H, V)
    if packed:
        pad = torch.full((B, T, 8), float("nan"), device="cuda")
        wide = torch.cat([q.flatten(2), k.flatten(2), v.flatten(2), pad], -1).to(dtype)
        q, k, v, _ = wide.split([Hk * K, Hk * K, H * V, 8], -1)
        q, k, v = q.unflatten(-1, (Hk, K)), k.unflatten(-1, (Hk, K)), v.unflatten(-1, (H, V))
    else:
        q, k, v = q.to(dtype), k.to(dtype), v.to(dtype)
    tau = torch.exp(torch.linspace(0.7, 6.0, H, device="cuda"))
    g = -(U.rand(seed + 3, B, T, H).abs() + 0.2) / tau
    beta = torch.sigmoid(U.rand(seed + 4, B, T, H))
    return dict(q=q, k=k, v=v, g=g, beta=beta, h0=U.rand(seed + 5, n or B, H, V, K, scale=0.3) if state else None)


def host(t):
    return {n: U.f64(v) for n, v in t.items()}
