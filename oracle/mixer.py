"""Plain fp64 numpy definitions of the gated delta rule with its gradient and of
the channels-last group norm with its gradient.  Written from the formulas, one
step after the other; test infrastructure, shares nothing with the HIP path."""
from __future__ import annotations

import numpy as np


def sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def _shared(t, heads):
    """(B, T, Hk, K) as the value heads see it: (B, T, heads, K)."""
    return np.repeat(np.asarray(t, np.float64), heads // t.shape[2], axis=2)


def delta_rule(q, k, v, g, beta, scale, h0=None):
    """y (B, T, H, V) and the states before each step and behind the last one,
    (T + 1, B, H, V, K)."""
    v = np.asarray(v, np.float64)
    B, T, H, V = v.shape
    q, k = _shared(q, H), _shared(k, H)
    K = q.shape[-1]
    s = np.zeros((B, H, V, K)) if h0 is None else np.array(h0, np.float64)
    y, states = np.empty_like(v), np.empty((T + 1, B, H, V, K))
    for t in range(T):
        states[t] = s
        s = np.exp(g[:, t])[..., None, None] * s
        r = v[:, t] - np.einsum("bhvk,bhk->bhv", s, k[:, t])
        s = s + (beta[:, t][..., None] * r)[..., None] * k[:, t][:, :, None]
        y[:, t] = scale * np.einsum("bhvk,bhk->bhv", s, q[:, t])
    states[T] = s
    return y, states


def delta_rule_bwd(q, k, v, g, beta, scale, dy, h0=None, dlast=None):
    """dict of dq, dk (summed over shared heads), dv, dg, dbeta, dh0, and of the
    sizes of what dg and dbeta are sums of (dg_terms, dbeta_terms)."""
    v, dy = np.asarray(v, np.float64), np.asarray(dy, np.float64)
    B, T, H, V = v.shape
    kheads = q.shape[2]
    _, states = delta_rule(q, k, v, g, beta, scale, h0)
    q, k = _shared(q, H), _shared(k, H)
    ds = np.zeros_like(states[0]) if dlast is None else np.array(dlast, np.float64)
    o = dict(dq=np.empty_like(q), dk=np.empty_like(k), dv=np.empty_like(v), dg=np.empty((B, T, H)), dbeta=np.empty((B, T, H)),
             dg_terms=np.empty((B, T, H)), dbeta_terms=np.empty((B, T, H)))
    for t in range(T - 1, -1, -1):
        kt, qt, a, b = k[:, t], q[:, t], np.exp(g[:, t])[..., None, None], beta[:, t][..., None]
        dec = a * states[t]
        r = v[:, t] - np.einsum("bhvk,bhk->bhv", dec, kt)
        s = states[t + 1]
        dyt = scale * dy[:, t]
        o["dq"][:, t] = np.einsum("bhvk,bhv->bhk", s, dyt)
        ds = ds + dyt[..., None] * qt[:, :, None]
        du = np.einsum("bhvk,bhk->bhv", ds, kt)
        dr = b * du
        write, read = np.einsum("bhvk,bhv->bhk", ds, b * r), np.einsum("bhvk,bhv->bhk", dec, dr)
        o["dk"][:, t], o["dv"][:, t] = write - read, dr
        o["dbeta"][:, t] = (du * r).sum(-1)
        o["dbeta_terms"][:, t] = np.sqrt((du * du).sum(-1) * (r * r).sum(-1))
        o["dg_terms"][:, t] = np.abs((qt * o["dq"][:, t]).sum(-1)) + np.abs((kt * write).sum(-1)) + np.abs((kt * read).sum(-1))
        ds = ds - dr[..., None] * kt[:, :, None]
        o["dg"][:, t] = (ds * dec).sum((-1, -2))
        ds = a * ds
    for n in ("dq", "dk"):
        o[n] = o[n].reshape(B, T, kheads, H // kheads, -1).sum(3)
    o["dh0"] = ds
    return o


def group_norm(x, groups, weight=None, bias=None, z=None, silu=False, eps=1e-5):
    """y, mean, rstd of x (N, R, C)."""
    x = np.asarray(x, np.float64)
    N, R, C = x.shape
    xg = x.reshape(N, R, groups, C // groups)
    mean = xg.mean((1, 3))
    var = ((xg - mean[:, None, :, None]) ** 2).mean((1, 3))
    rstd = 1.0 / np.sqrt(var + eps)
    return group_norm_at(x, mean, rstd, weight, bias, z, silu), mean, rstd


def _normalised(x, mean, rstd):
    rep = lambda t: np.repeat(np.asarray(t, np.float64), x.shape[-1] // t.shape[-1], axis=-1)[:, None]
    return (np.asarray(x, np.float64) - rep(mean)) * rep(rstd), rep(rstd)


def group_norm_at(x, mean, rstd, weight=None, bias=None, z=None, silu=False):
    n, _ = _normalised(x, mean, rstd)
    a = n * (1.0 if weight is None else weight) + (0.0 if bias is None else bias)
    y = a * sigmoid(a) if silu else a
    return y if z is None else y * z * sigmoid(z)


def group_norm_bwd(dy, x, mean, rstd, weight=None, bias=None, z=None, silu=False):
    """dict of dx, dz, dweight, dbias, and the sizes of what the sums add up
    (dweight_terms, dbias_terms: sqrt of the sum of squares)."""
    N, R, C = x.shape
    groups = mean.shape[-1]
    n, rep_rstd = _normalised(x, mean, rstd)
    w = np.ones(C) if weight is None else np.asarray(weight, np.float64)
    a = n * w + (0.0 if bias is None else bias)
    sa = sigmoid(a)
    da, out = np.asarray(dy, np.float64), {}
    if z is not None:
        z = np.asarray(z, np.float64)
        sz = sigmoid(z)
        out["dz"] = da * (a * sa if silu else a) * sz * (1.0 + z * (1.0 - sz))
        da = da * z * sz
    if silu:
        da = da * sa * (1.0 + a * (1.0 - sa))
    out.update(dweight=(da * n).sum((0, 1)), dbias=da.sum((0, 1)), dweight_terms=np.sqrt(((da * n) ** 2).sum((0, 1))),
               dbias_terms=np.sqrt((da ** 2).sum((0, 1))))
    gm = lambda t: np.repeat(t.reshape(N, R, groups, C // groups).mean((1, 3)), C // groups, axis=-1)[:, None]
    out["dx"] = rep_rstd * (w * da - gm(w * da) - n * gm(w * da * n))
    return out
