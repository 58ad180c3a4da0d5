"""Plain fp64 numpy definitions of the gated recurrent block's operators: the
gated linear recurrence and its gradient, the RMS norm with the residual's
addition (with its 8-bit form) and its gradient, the global gradient norm and
clipping.  Written from the formulas, one step after the other; test
infrastructure, shares nothing with the HIP path.

Beside each result the functions can return a bound on the rounding error of an
fp32 evaluation of the same formulas (`bounds=True`), from first-order error
propagation: every fp32 operation is off by at most U = 2^-24 relative, and
errors pass through the recurrence as the values do (the same recurrence run on
absolute values)."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
# fp32's smallest normal number.  exp(-|v|) below it comes out as 0 (the
# hardware's exponential returns no subnormal results), so the smaller side of a
# gate, exp(-|v|) / (1 + exp(-|v|)), is off by up to TINY absolutely beside its
# relative error, and so is whatever it multiplies, times that factor: at v = -88
# the gate's side is 6.1e-39 < TINY = 1.2e-38, and with a factor of 2.9 the
# product 1.7e-38 is lost whole.
TINY = 2.0 ** -126


def sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def _gate(g, bias):
    with np.errstate(over="ignore"):
        v = g if bias is None else g + bias
    return v, sigmoid(v), sigmoid(-v)


def _gate_units(v):
    """Relative error of an fp32 sigmoid in units of U: the sum g + bias is off
    by |v| U, which shifts the exponential by as much relatively; the
    exponential, the sum, the quotient and the complement add 12 U at most.
    Past |v| = 128 both sides are exactly 0 and 1 in fp32."""
    return np.minimum(np.abs(v), 128.0) + 12.0


def gated_scan(x, g, z=None, gate_bias=None, h0=None, bounds=False):
    """y, last (and the bounds of both)."""
    x, g = np.asarray(x, np.float64), np.asarray(g, np.float64)
    Bt, T, D = x.shape
    v, a, s = _gate(g, gate_bias)
    h = np.zeros((Bt, D)) if h0 is None else np.array(h0, np.float64)
    H, E = np.abs(h), np.zeros((Bt, D))
    hs, es = np.empty_like(x), np.empty_like(x)
    # per step: the gate's error, one rounding of (1 - a) x, one of the sum, one
    # of the decay products that carry a state over several steps, and a quarter
    # for the sums of the tiles' hand-over (under 32 of them per 128 steps)
    k = _gate_units(v) + 4.0
    for t in range(T):
        h = a[:, t] * h + s[:, t] * x[:, t]
        Hn = a[:, t] * H + s[:, t] * np.abs(x[:, t])
        E = a[:, t] * E + k[:, t] * U * Hn + TINY * (H + np.abs(x[:, t]))
        H = Hn
        hs[:, t], es[:, t] = h, E
    y, ey = hs, es
    if z is not None:
        z = np.asarray(z, np.float64)
        sl = z * sigmoid(z)
        y = hs * sl
        ey = np.abs(sl) * (es + np.abs(hs) * (_gate_units(z) + 2.0) * U)
    return (y, h, ey, E) if bounds else (y, h)


def _bias_additions(batch, T):
    """Additions on any path of dgate_bias: a wave's 16 steps, a tile's 8 waves,
    every 64th of the tiles' sums, the 64 stripes of those by halves."""
    return 16 + 8 + -(-batch * -(-T // 128) // 64) + 6


def gated_scan_bwd(x, g, dout, z=None, gate_bias=None, h0=None, dlast=None, bounds=False):
    """dict of dx, dg, dz, dgate_bias, dh0 (and one of their bounds)."""
    x, g, dout = (np.asarray(t, np.float64) for t in (x, g, dout))
    Bt, T, D = x.shape
    v, a, s = _gate(g, gate_bias)
    k = _gate_units(v) + 4.0
    hb, eb = np.empty_like(x), np.empty_like(x)          # before each step, and its bound
    hh, eh = np.empty_like(x), np.empty_like(x)          # after
    h = np.zeros((Bt, D)) if h0 is None else np.array(h0, np.float64)
    H, E = np.abs(h), np.zeros((Bt, D))
    for t in range(T):
        hb[:, t], eb[:, t] = h, E
        h = a[:, t] * h + s[:, t] * x[:, t]
        Hn = a[:, t] * H + s[:, t] * np.abs(x[:, t])
        E = a[:, t] * E + k[:, t] * U * Hn + TINY * (H + np.abs(x[:, t]))
        H = Hn
        hh[:, t], eh[:, t] = h, E
    d, ed = dout, np.zeros_like(dout)
    out, bd = {}, {}
    if z is not None:
        z = np.asarray(z, np.float64)
        sg = sigmoid(z)
        d = dout * z * sg
        ed = np.abs(d) * (_gate_units(z) + 2.0) * U
        dsilu = sg * (1.0 + z * (1.0 - sg))
        out["dz"] = dout * hh * dsilu
        bd["dz"] = np.abs(dout) * (eh * np.abs(dsilu) + np.abs(hh) * sg * (1.0 + np.abs(z) * (1.0 - sg))
                                   * (2.0 * _gate_units(z) + 6.0) * U)
    e = np.zeros((Bt, D)) if dlast is None else np.array(dlast, np.float64)
    A, F = np.abs(e), np.zeros((Bt, D))
    es, fs = np.empty_like(x), np.empty_like(x)
    for t in range(T - 1, -1, -1):
        e, A = d[:, t] + e, np.abs(d[:, t]) + A
        F = F + ed[:, t] + U * A
        es[:, t], fs[:, t] = e, F
        F = a[:, t] * (F + k[:, t] * U * A) + TINY * A
        e, A = a[:, t] * e, a[:, t] * A
    with np.errstate(invalid="ignore"):
        dg = es * (hb - x) * a * s
    out.update(dx=s * es, dg=dg, dgate_bias=dg.sum((0, 1)), dh0=e)
    if not bounds:
        return out
    w = np.abs(a * s)
    bd["dx"] = s * fs + np.abs(s * es) * (k + 2.0) * U + TINY * np.abs(es)
    bd["dg"] = w * (fs * np.abs(hb - x) + np.abs(es) * (eb + U * np.abs(hb - x))) + np.abs(dg) * (2.0 * k + 6.0) * U \
        + TINY * np.abs(es * (hb - x))
    bd["dgate_bias"] = bd["dg"].sum((0, 1)) + _bias_additions(Bt, T) * U * np.abs(dg).sum((0, 1))
    bd["dh0"] = F
    return out, bd


def _units(dim):
    """Additions on any path of a row's sum: at most 16 per register lane chain
    of dim / 64 values, and 16 across lanes and waves."""
    return dim / 64.0 + 24.0


def _weight_additions(rows):
    """Additions on any path of dweight: the rows that a lane walks (every 512th at
    most), up to 32 rows side by side in a workgroup, up to 1024 workgroups' sums,
    every 64th, and the stripes by halves."""
    return -(-rows // 512) + 32 + 16 + 6


def add_rms_norm(x, weight, residual=None, eps=1e-5, bounds=False):
    """r, y (and y's bound; r's is U |r|)."""
    x, w = np.asarray(x, np.float64), np.asarray(weight, np.float64)
    r = x if residual is None else x + np.asarray(residual, np.float64)
    y = r / np.sqrt((r * r).mean(-1, keepdims=True) + eps) * w
    return (r, y, np.abs(y) * (0.5 * _units(r.shape[-1]) + 10.0) * U) if bounds else (r, y)


def add_rms_norm_scale(y):
    return np.maximum(np.abs(y).max(-1) / 448.0, 2.0 ** -126)


def add_rms_norm_bwd(dy, r, weight, dresidual=None, eps=1e-5, bounds=False):
    """dr, dweight (and their bounds)."""
    dy, r, w = (np.asarray(t, np.float64) for t in (dy, r, weight))
    rstd = 1.0 / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
    n = r * rstd
    c = (n * w * dy).mean(-1, keepdims=True)
    dr = rstd * (w * dy - n * c)
    add = 0.0 if dresidual is None else np.asarray(dresidual, np.float64)
    if not bounds:
        return dr + add, (dy * n).sum(0)
    k = 2.0 * _units(r.shape[-1]) + 16.0
    mag = rstd * (np.abs(w * dy) + np.abs(n) * np.abs(n * w * dy).mean(-1, keepdims=True))
    bdr = mag * k * U + np.abs(dr + add) * U
    bdw = np.abs(dy * n).sum(0) * (0.5 * k + _weight_additions(len(r))) * U
    return dr + add, (dy * n).sum(0), bdr, bdw


def clip(grads, max_norm, eps=1e-6):
    """norm, coefficient."""
    norm = np.sqrt(sum(float((np.asarray(g, np.float64) ** 2).sum()) for g in grads))
    return norm, min(1.0, max_norm / (norm + eps))
