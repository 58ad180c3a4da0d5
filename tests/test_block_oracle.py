"""The gated recurrent block's fp64 definitions (oracle/recurrent_block.py)
against facts of their own: a hand-worked chain, the unrolled sum, continuation,
the gates' limits, central differences of the forward, torch's float64 autograd."""
import numpy as np
import pytest
import torch

from oracle import recurrent_block as R


def rand(rng, *shape):
    return rng.standard_normal(shape)


def test_hand_worked_chain():
    # a = 1/2, 1/4 (gates 0 and -log 3), x = 2, 4, h0 = 1: h = 1.5, then 0.375 + 3 = 3.375
    x = np.array([2.0, 4.0]).reshape(1, 2, 1)
    g = np.array([0.0, -np.log(3.0)]).reshape(1, 2, 1)
    y, last = R.gated_scan(x, g, h0=np.ones((1, 1)))
    assert np.allclose(y[0, :, 0], [1.5, 3.375], rtol=1e-15) and np.allclose(last, 3.375, rtol=1e-15)


def test_unrolled_sum():
    rng = np.random.default_rng(1)
    x, g, b, h0 = rand(rng, 2, 9, 3), rand(rng, 2, 9, 3), rand(rng, 3), rand(rng, 2, 3)
    a = 1.0 / (1.0 + np.exp(-(g + b)))
    y, _ = R.gated_scan(x, g, gate_bias=b, h0=h0)
    for t in range(9):
        want = np.prod(a[:, :t + 1], 1) * h0
        for s in range(t + 1):
            want = want + np.prod(a[:, s + 1:t + 1], 1) * (1.0 - a[:, s]) * x[:, s]
        assert np.allclose(y[:, t], want, rtol=1e-12, atol=1e-13)


def test_infinite_gates_keep_and_restart():
    rng = np.random.default_rng(2)
    x, g, h0 = rand(rng, 1, 6, 4), rand(rng, 1, 6, 4), rand(rng, 1, 4)
    g[:, 2:4] = np.inf
    y, _ = R.gated_scan(x, g, h0=h0)
    assert np.array_equal(y[:, 2], y[:, 1]) and np.array_equal(y[:, 3], y[:, 1])
    g[:, 4] = -np.inf
    y, _ = R.gated_scan(x, g, h0=h0)
    assert np.array_equal(y[:, 4], x[:, 4])
    assert np.array_equal(R.gated_scan(x[:, 4:], g[:, 4:])[0], y[:, 4:])


def test_continuation():
    rng = np.random.default_rng(3)
    x, g, z = (rand(rng, 2, 11, 3) for _ in range(3))
    y, last = R.gated_scan(x, g, z)
    y1, l1 = R.gated_scan(x[:, :4], g[:, :4], z[:, :4])
    y2, l2 = R.gated_scan(x[:, 4:], g[:, 4:], z[:, 4:], h0=l1)
    assert np.array_equal(np.concatenate([y1, y2], 1), y) and np.array_equal(l2, last)


@pytest.mark.parametrize("with_z", [False, True])
def test_gated_gradient_by_differences(with_z):
    rng = np.random.default_rng(4)
    t = dict(x=rand(rng, 2, 5, 2), g=rand(rng, 2, 5, 2), gate_bias=rand(rng, 2), h0=rand(rng, 2, 2))
    if with_z:
        t["z"] = rand(rng, 2, 5, 2)
    dout, dlast = rand(rng, 2, 5, 2), rand(rng, 2, 2)

    def loss(**kw):
        y, last = R.gated_scan(**kw)
        return (y * dout).sum() + (last * dlast).sum()

    got = R.gated_scan_bwd(dout=dout, dlast=dlast, **t)
    for name, value in t.items():
        for i in np.ndindex(value.shape):
            lo, hi = value.copy(), value.copy()
            lo[i] -= 1e-5
            hi[i] += 1e-5
            want = (loss(**{**t, name: hi}) - loss(**{**t, name: lo})) / 2e-5
            assert abs(got["d" + name][i] - want) < 1e-8, (name, i)


def test_norm_against_autograd():
    rng = np.random.default_rng(5)
    x, res, w, dy, dr = rand(rng, 4, 7), rand(rng, 4, 7), rand(rng, 7), rand(rng, 4, 7), rand(rng, 4, 7)
    tx, tr, tw = (torch.from_numpy(v).requires_grad_() for v in (x, res, w))
    r = tx + tr
    y = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + 1e-5) * tw
    ((y * torch.from_numpy(dy)).sum() + (r * torch.from_numpy(dr)).sum()).backward()
    ro, yo = R.add_rms_norm(x, w, res)
    assert np.allclose(ro, r.detach().numpy(), rtol=1e-15) and np.allclose(yo, y.detach().numpy(), rtol=1e-12)
    dro, dwo = R.add_rms_norm_bwd(dy, ro, w, dr)
    assert np.allclose(dro, tx.grad.numpy(), rtol=1e-11, atol=1e-13) and np.allclose(dro, tr.grad.numpy(), rtol=1e-11, atol=1e-13)
    assert np.allclose(dwo, tw.grad.numpy(), rtol=1e-11, atol=1e-13)


def test_scale_floor():
    assert R.add_rms_norm_scale(np.zeros((1, 3)))[0] == 2.0 ** -126
    assert R.add_rms_norm_scale(np.array([[1.0, -896.0]]))[0] == 2.0


def test_clip_by_hand():
    norm, coef = R.clip([np.array([3.0]), np.array([[4.0]])], 1.0, eps=0.0)
    assert norm == 5.0 and coef == 0.2
    assert R.clip([np.array([3.0])], 10.0)[1] == 1.0


def test_bounds_cover_an_fp32_evaluation():
    """The stated rounding bounds hold for a plain fp32 evaluation, with room
    of at least 4 (they are worst cases) and at most 10^4 (they are no blanket)."""
    rng = np.random.default_rng(6)
    f = np.float32
    x, g, b = (rng.standard_normal(s).astype(f) for s in ((1, 300, 64), (1, 300, 64), (64,)))
    y, _, ey, _ = R.gated_scan(x, g, gate_bias=b, bounds=True)
    h = np.zeros((1, 64), f)
    worst = 0.0
    for t in range(300):
        v = g[:, t] + b
        a, s = f(1) / (f(1) + np.exp(-v)), f(1) / (f(1) + np.exp(v))
        h = a * h + s * x[:, t]
        worst = max(worst, float((np.abs(h - y[:, t]) / ey[:, t]).max()))
    assert 1e-4 < worst < 0.25


def column_sums(parts):
    """fp32 sums of the columns: every 64th row one after the other, then the 64 stripes by halves."""
    rows, dim = parts.shape
    s = np.zeros((-(-rows // 64) * 64, dim), np.float32)
    s[:rows] = parts
    s = s.reshape(-1, 64, dim)
    acc = np.zeros((64, dim), np.float32)
    for r in s:
        acc = acc + r
    while len(acc) > 1:
        acc = acc[0::2] + acc[1::2]
    return acc[0]


def test_bias_bound_counts_the_additions_of_a_large_batch():
    """One large value and a thousand small ones in every stripe: each small one is lost where it is added."""
    B = 65535
    dg = np.where(np.arange(B) < 64, 1.0, 0.99 * 2.0 ** -24)
    x, g = -np.ones((B, 1, 1)), np.zeros((B, 1, 1))            # a = 1 - a = 1/2, dg = dout / 4
    want, bound = R.gated_scan_bwd(x, g, 4.0 * dg.reshape(B, 1, 1), bounds=True)
    assert np.allclose(want["dgate_bias"], dg.sum(), rtol=1e-12)
    got = column_sums(dg.astype(np.float32).reshape(B, 1))
    assert 0.5 * bound["dgate_bias"] < np.abs(got - want["dgate_bias"]) < bound["dgate_bias"]


def test_weight_bound_counts_the_additions_of_many_rows():
    rows = 400000
    dy = np.where(np.arange(rows) < 512, 1.0, 0.99 * 2.0 ** -24).reshape(rows, 1)
    _, want, _, bound = R.add_rms_norm_bwd(dy, np.ones((rows, 1)), np.ones(1), eps=0.0, bounds=True)
    acc = np.zeros((512, 1), np.float32)                         # a workgroup takes every 512th row
    for i in range(0, rows, 512):
        v = dy[i:i + 512].astype(np.float32)
        acc[:len(v)] = acc[:len(v)] + v
    assert 0.5 * bound[0] < abs(column_sums(acc)[0] - want[0]) < bound[0]


def test_small_sizes_have_small_bounds():
    """The additions are counted, not a blanket: 300 steps of two sequences take 31 of them on a path, 40 rows 55."""
    assert R._bias_additions(2, 300) == 31 and R._weight_additions(40) == 55


def test_differences_along_the_signs_reject_a_gradient_one_percent_off():
    from block_util import along_its_signs
    f = lambda seed, *shape: torch.randn(shape, generator=torch.Generator().manual_seed(seed)).double().numpy()
    B, T, D = 2, 300, 64
    t = dict(x=f(0, B, T, D), g=f(1, B, T, D), z=f(2, B, T, D), gate_bias=np.abs(f(5, D)) * 2.5, h0=f(6, B, D))
    dout, dlast = f(90, B, T, D), f(91, B, D)
    got = R.gated_scan_bwd(t["x"], t["g"], dout, t["z"], t["gate_bias"], t["h0"], dlast)
    _, _, ey, el = R.gated_scan(**t, bounds=True)
    noise = np.sqrt(((ey * dout) ** 2).sum() + ((el * dlast) ** 2).sum())

    def loss(a):
        y, last = R.gated_scan(**a)
        return (y * dout).sum() + (last * dlast).sum()

    for name in t:
        off, allowed = along_its_signs(loss, t, name, got["d" + name], 0.02, noise)
        assert off <= allowed, name
        for factor in (0.99, 1.01):
            off, allowed = along_its_signs(loss, t, name, got["d" + name] * factor, 0.02, noise)
            assert off > allowed, (name, factor)
