"""The channels-last group norm on the GPU against its fp64 definition.

Tolerances.  mean and rstd: with one row a group's sums are fp32, at most
D / 64 + 12 additions on any path, so the mean is off by (D / 64 + 12) U of
mean|x|, and rstd by as much relatively, plus 8 U of its own operations; over
several rows up to 8 neighbouring values are added in fp32, the rest in fp64: 8 U of
mean|x| and two roundings.  An element: (x - mean)
rstd is off by U (|x| + |mean|) rstd for the difference, the statistics' errors and
4 roundings; the activation multiplies that by its slope (at most 1.1, twice with
the gate) and adds its own error, an exponential's, a sum's and a quotient's:
(|argument| + 12) U relative."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_util as U
from oracle import mixer as M

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from selective_scan_ssm_amd import _lib, ops
    _lib.load()
    return ops


def inputs(N, R, C, dtype, gate=False, affine=True, strided=False, seed=0, offset=0.5):
    x = U.rand(seed, N, R, C) * (0.5 + U.rand(seed + 1, C).abs()) + offset * U.rand(seed + 2, C)
    z = U.rand(seed + 3, N, R, C) if gate else None
    if strided:
        wide = torch.cat([x, x if z is None else z, torch.full((N, R, 8), float("nan"), device="cuda")], -1).to(dtype)
        x, z = wide[..., :C], wide[..., C:2 * C] if gate else None
    else:
        x, z = x.to(dtype), None if z is None else z.to(dtype)
    w, b = (1.0 + 0.2 * U.rand(seed + 4, C), 0.3 * U.rand(seed + 5, C)) if affine else (None, None)
    return dict(x=x, z=z, weight=w, bias=b)


def bound_of(x, mean, rstd, groups, w, b, z, silu):
    """The bound of y's fp32 evaluation, and of n's."""
    N, R, C = x.shape
    D = C // groups
    rep = lambda t: np.repeat(t, D, axis=-1)[:, None]
    k = (D / 64.0 + 12.0) if R == 1 else 10.0
    ax = np.abs(x).reshape(N, R, groups, D).mean((1, 3))
    n = (x - rep(mean)) * rep(rstd)
    en = EPS * ((np.abs(x) + np.abs(rep(mean)) + k * rep(ax)) * rep(rstd) + (2.0 * k + 12.0) * np.abs(n))
    w = np.ones(C) if w is None else np.abs(w)
    a = np.abs(n) * w + (0.0 if b is None else np.abs(b))
    ea = en * w + 3.0 * EPS * a
    ey = 1.1 * ea + (EPS * (a + 12.0) * a if silu else 0.0)
    if z is not None:
        sz = np.abs(z * M.sigmoid(z))
        ey = ey * sz + a * sz * (np.abs(z) + 14.0) * EPS
    return ey, en


def check(ops, t, groups, silu=False, eps=1e-5, seed=40, shape=None, grads=True):
    x = t["x"]
    N, C = x.shape[0], x.shape[-1]
    R = x[0].numel() // C
    act = "silu" if silu else None
    y, guard = U.guarded(tuple(x.shape), x.dtype)
    _, mean, rstd = ops.group_norm(x, groups, t["weight"], t["bias"], z=t["z"], activation=act, eps=eps, return_stats=True, out=y)
    torch.cuda.synchronize()
    guard()
    f = lambda a: None if a is None else U.f64(a).reshape(N, R, C)
    xo, zo, w, b = f(x), f(t["z"]), U.f64(t["weight"]), U.f64(t["bias"])
    yo, mo, ro = M.group_norm(xo, groups, w, b, zo, silu, eps)
    D = C // groups
    k = (D / 64.0 + 12.0) if R == 1 else 10.0
    ax = np.abs(xo).reshape(N, R, groups, D).mean((1, 3))
    assert (np.abs(U.f64(mean) - mo) <= k * EPS * ax + 2.0 ** -126).all()
    # rstd: of the sum of squares, and the mean's own error enters squared beside eps
    assert (np.abs(U.f64(rstd) - ro) <= (k + 8.0) * EPS * ro + (k * EPS * ax * ro) ** 2 * ro).all()
    ey, en = bound_of(xo, mo, ro, groups, w, b, zo, silu)
    U.close(y.reshape(N, R, C), yo, ey, "y")
    if not grads:
        return y
    dy = U.rand(seed, *x.shape, dtype=x.dtype)
    got = ops.group_norm_bwd(dy, x, mean, rstd, groups, t["weight"], t["bias"], z=t["z"], activation=act)
    torch.cuda.synchronize()
    m, r = U.f64(mean), U.f64(rstd)
    want = M.group_norm_bwd(f(dy), xo, m, r, w, b, zo, silu)
    rep = lambda q: np.repeat(q, D, axis=-1)[:, None]
    n = (xo - rep(m)) * rep(r)
    wa = np.ones(C) if w is None else np.abs(w)
    a = np.abs(n) * wa + (0.0 if b is None else np.abs(b))
    # da's bound: the slopes' own errors, and theirs by a (the activation's second derivative is under 0.6)
    u = EPS * ((np.abs(xo) + np.abs(rep(m))) * rep(r) + 6.0 * np.abs(n))
    g = np.abs(f(dy))
    if zo is not None:
        sz = M.sigmoid(zo)
        if "dz" in want:
            slope = np.abs(sz * (1.0 + zo * (1.0 - sz)))
            val = a if not silu else np.abs(a)
            bz = g * (1.1 * (u * wa + 3 * EPS * a) * slope + val * (slope + sz * np.abs(zo)) * (np.abs(zo) + (a if silu else 0.0) + 28.0) * EPS)
            U.close(got["dz"].reshape(N, R, C), want["dz"], bz, "dz")
        g = g * np.abs(zo * sz) * (1.0 + (np.abs(zo) + 14.0) * EPS)
        ez = np.abs(zo) + 14.0
    else:
        ez = 0.0
    da_abs = g * 1.1 if silu else g
    bda = da_abs * (ez + ((2.0 * a + 28.0) if silu else 0.0)) * EPS + (0.6 * g * (u * wa + 3 * EPS * a) if silu else 0.0)
    # column sums of N R values: fp32, the additions on any path (a thread's rows, 256 threads or 4 waves, 64 runs' stripes)
    adds = N * R / 64.0 + 200.0
    if w is not None:
        U.close(got["dweight"], want["dweight"], (bda * np.abs(n) + da_abs * u).sum((0, 1)) + adds * EPS * (da_abs * np.abs(n)).sum((0, 1)), "dweight")
    else:
        assert got["dweight"] is None
    if b is not None:
        U.close(got["dbias"], want["dbias"], bda.sum((0, 1)) + adds * EPS * da_abs.sum((0, 1)), "dbias")
    gm = lambda q: rep(q.reshape(N, R, groups, D).mean((1, 3)))
    kk = (D / 64.0 + 12.0) if R == 1 else R / 64.0 + 200.0
    t1, t2 = wa * da_abs, wa * da_abs * np.abs(n)
    bdx = rep(r) * (wa * bda + gm(wa * bda) + np.abs(n) * gm(wa * bda * np.abs(n) + t1 * u) + u * gm(t2)
                    + EPS * (8.0 * t1 + (kk + 8.0) * (gm(t1) + np.abs(n) * gm(t2))))
    U.close(got["dx"].reshape(N, R, C), want["dx"], bdx, "dx")
    return y


# one row to a statistic: a lane to several chunks of a wave, odd widths, groups that fill a wave in part
ROWS = [(1, 8, 1), (3, 8, 8), (5, 24, 3), (7, 96, 1), (4, 130, 5), (33, 640, 5), (2, 321, 1), (3, 321, 107), (9, 1536, 12), (5, 5120, 40),
        (3, 4096, 2), (2, 2080, 1), (300, 64, 16), (2, 1000, 1), (5000, 16, 2)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,C,G", ROWS)
def test_one_row(ops, N, C, G, dtype):
    silu, gate = (N + C) % 2 == 0, C % 3 != 0
    check(ops, inputs(N, 1, C, DT[dtype], gate=gate, affine=C % 5 != 0, strided=N % 2 == 1, seed=C), G, silu)


# several rows: one to many runs, groups narrower and wider than a workgroup's lanes
MAPS = [(1, 2, 8, 1), (2, 3, 24, 3), (3, 196, 96, 8), (1, 1000, 6, 2), (2, 49, 320, 32), (1, 64, 2304, 4), (4, 9, 33, 11), (2, 777, 192, 32),
        (1, 5, 5000, 1), (1, 4096, 64, 4), (40, 16, 16, 16), (2, 30, 9000, 3), (1, 3, 4098, 2),
        # around the most rows of a batch entry whose groups stay in registers, forward and gradient
        (2, 256, 64, 4), (1, 257, 64, 4), (2, 512, 64, 8), (1, 513, 64, 8), (3, 600, 20, 2),
        # few rows of many groups
        (5, 2, 1536, 12), (3, 4, 40, 40), (2, 2, 2056, 2), (1, 3, 1000, 500)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,R,C,G", MAPS)
def test_maps(ops, N, R, C, G, dtype):
    check(ops, inputs(N, R, C, DT[dtype], gate=R % 2 == 0, affine=C % 7 != 0, strided=R % 3 == 0, seed=R), G, silu=C % 2 == 0)


def test_axes_between(ops):
    """(batch, height, width, dim) is (batch, height * width, dim)."""
    t = inputs(2, 35, 64, torch.float32)
    y = check(ops, t, 8, silu=True)
    y4 = ops.group_norm(t["x"].view(2, 5, 7, 64), 8, t["weight"], t["bias"], activation="silu")
    assert y4.shape == (2, 5, 7, 64) and torch.equal(y4.view(2, 35, 64), y)
    assert torch.equal(ops.group_norm(t["x"][:, 0].contiguous(), 8), ops.group_norm(t["x"][:, :1].contiguous(), 8)[:, 0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R", [1, 100])
def test_unaligned_bases(ops, R, dtype):
    """Addresses and strides that allow no wide access."""
    N, C = 3, 64
    wide = U.rand(5, N, R, C + 1, dtype=DT[dtype])
    t = inputs(N, R, C, DT[dtype], gate=True)
    t["x"], t["z"] = wide[..., 1:], U.rand(6, N, R, C + 3, dtype=DT[dtype])[..., 2:C + 2]
    check(ops, t, 4, silu=True)


@pytest.mark.parametrize("R", [1, 50, 3000])
def test_far_means(ops, R):
    """A mean of some thousand standard deviations."""
    t = inputs(2, R, 128, torch.float32, offset=0.0)
    t["x"] = t["x"] + 4096.0
    check(ops, t, 4)


@pytest.mark.parametrize("R", [50, 3000])
def test_first_values_far_from_the_rest(ops, R):
    t = inputs(2, R, 128, torch.float32)
    t["x"][:, :8] = 3e4
    check(ops, t, 4)


@pytest.mark.parametrize("R", [1, 20])
def test_constant_groups_and_large_arguments(ops, R):
    t = inputs(2, R, 64, torch.float32, gate=True)
    t["x"][0, :, :16] = 3.25
    t["bias"][20:30], t["bias"][30:40] = 200.0, -200.0
    t["z"][1, :, ::5], t["z"][1, :, 1::5] = 300.0, -300.0
    check(ops, t, 4, silu=True)


def test_a_nan_stays_in_its_group(ops):
    for R in (1, 30):
        t = inputs(3, R, 64, torch.float32)
        clean = ops.group_norm(t["x"], 4, t["weight"], t["bias"])
        t["x"][1, 0, 20] = float("nan")
        y = ops.group_norm(t["x"], 4, t["weight"], t["bias"])
        bad = torch.isnan(y)
        assert bool(bad[1, :, 16:32].all()) and int(bad.sum()) == R * 16 and torch.equal(y[~bad], clean[~bad])


def test_empty(ops):
    w = torch.ones(8, device="cuda")
    for shape in ((0, 5, 8), (3, 0, 8)):
        x = torch.empty(shape, device="cuda")
        y, mean, rstd = ops.group_norm(x, 2, w, w, return_stats=True)
        got = ops.group_norm_bwd(x, x, mean, rstd, 2, w, w)
        assert y.shape == shape and not bool(got["dweight"].any()) and not bool(got["dbias"].any())
        assert bool(torch.isnan(mean).all()) and bool(torch.isnan(rstd).all())


def test_many_groups_of_one_channel(ops):
    """Groups of one channel over more batch entries than a launch's second axis holds."""
    t = inputs(66000, 2, 16, torch.float32)
    y, mean, rstd = ops.group_norm(t["x"], 16, t["weight"], t["bias"], return_stats=True)
    m = t["x"].double().mean(1)
    assert float((mean.double() - m).abs().max()) <= 10 * EPS * float(t["x"].abs().max())
    again = ops.group_norm(t["x"][65990:], 16, t["weight"], t["bias"])
    assert torch.equal(again, y[65990:])


def test_large_batches_and_wide_offsets(ops):
    """More rows than workgroups; a tensor past 2^31 bytes."""
    t = inputs(70001, 1, 48, torch.bfloat16, gate=True)
    y = ops.group_norm(t["x"], 3, t["weight"], t["bias"], z=t["z"])
    part = {k: v[69990:] if k in "xz" else v for k, v in t.items()}
    assert torch.equal(ops.group_norm(part["x"].contiguous(), 3, part["weight"], part["bias"], z=part["z"].contiguous()), y[69990:])
    x = torch.zeros(3, 1 << 15, 1 << 14, dtype=torch.bfloat16, device="cuda")          # 3 GiB, 2^30 bytes to an entry
    x[2, -64:] = U.rand(1, 64, 1 << 14, dtype=torch.bfloat16)
    y, mean, rstd = ops.group_norm(x, 4, return_stats=True)
    n = (1 << 15) * (1 << 12)
    g = x[2, -64:].double().view(64, 4, 1 << 12)
    m = g.sum((0, 2)) / n
    v = (g * g).sum((0, 2)) / n - m * m
    assert torch.allclose(mean[2].double(), m, rtol=1e-6) and torch.allclose(rstd[2].double(), (v + 1e-5).rsqrt(), rtol=1e-6)
    want = ((g - m[:, None]) * (v + 1e-5).rsqrt()[:, None]).view(64, 1 << 14)
    assert torch.allclose(y[2, -64:].double(), want, rtol=2.0 ** -8, atol=1e-5)


@pytest.mark.parametrize("R", [1, 300])
def test_streams_graphs_and_repeats(ops, R):
    N, C, G = 64 if R == 1 else 3, 192, 12
    t = inputs(N, R, C, torch.bfloat16, gate=True)
    dy = U.rand(8, N, R, C, dtype=torch.bfloat16)

    def step():
        y, mean, rstd = ops.group_norm(t["x"], G, t["weight"], t["bias"], z=t["z"], activation="silu", return_stats=True)
        return [y, mean, rstd, *ops.group_norm_bwd(dy, t["x"], mean, rstd, G, t["weight"], t["bias"], z=t["z"], activation="silu").values()]

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for r in range(3):
        t["x"].copy_(U.rand(60 + r, N, R, C))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_refusals(ops):
    t = inputs(2, 4, 24, torch.float32, gate=True)
    x, w, b, z = t["x"], t["weight"], t["bias"], t["z"]
    for kw in (dict(x=x.half()), dict(x=x[0, 0]), dict(weight=w[:8]), dict(bias=b.bfloat16()), dict(z=z.bfloat16()), dict(z=z[:1]),
               dict(activation="gelu"), dict(x=x.cpu()), dict(x=x.transpose(1, 2)), dict(out=x[:1])):
        with pytest.raises(ValueError):
            ops.group_norm(**{**dict(x=x, groups=4, weight=w, bias=b, z=z), **kw})
    for groups in (0, 5, 48):
        with pytest.raises(RuntimeError):
            ops.group_norm(x, groups)
    with pytest.raises(RuntimeError):
        ops.group_norm(x, 4, eps=-1.0)
    mean = torch.zeros(2, 4, device="cuda")
    for kw in (dict(dy=x[:1]), dict(mean=mean[:1]), dict(rstd=mean.double())):
        with pytest.raises(ValueError):
            ops.group_norm_bwd(**{**dict(dy=x, x=x, mean=mean, rstd=mean, groups=4), **kw})
