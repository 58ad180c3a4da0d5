"""The RMS norm with the residual's addition on the GPU against its fp64
definition, within the rounding bounds derived beside it."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_util as U
from oracle import recurrent_block as R

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
TYPES = [(F32, F32), (BF16, BF16), (BF16, F32)]


@pytest.fixture(scope="module", autouse=True)
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from selective_scan_ssm_amd import _lib, ops
    _lib.load()
    return ops


def e4m3_half_step(v):
    """Half the distance between neighbours of e4m3 around |v| <= 448."""
    e = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6)))
    return 2.0 ** (e - 4)


def check_quant(q, scale, y, by):
    want = R.add_rms_norm_scale(y)
    rel = by.max(-1) / np.maximum(np.abs(y).max(-1), 1e-300) + 4 * R.U
    s = U.f64(scale)
    assert np.all(np.abs(s - want) <= want * rel), "scale"
    v = y / want[..., None]
    off = np.abs(U.f64(q) - v)
    # half a step of the format, plus the fp32 error of y / scale before it is rounded
    tol = e4m3_half_step(v) * (1 + 1e-6) + by / want[..., None] + np.abs(v) * (rel[..., None] + 4 * R.U)
    assert np.all(off <= tol), f"q: {np.max(off - tol)}"


SIZES = [(1, 1), (3, 2), (5, 63), (2, 64), (7, 65), (4, 130), (9, 256), (3, 257), (130, 768), (5, 1000), (17, 1536), (3, 2049),
         (1000, 8), (37, 16), (5, 24), (130, 32), (67, 128), (33, 200), (21, 1540), (9, 100), (3, 31), (259, 17), (33, 2560), (2, 4097), (6, 5120), (2, 8192), (1, 10001), (2, 16384), (1, 32768), (1, 32767)]


@pytest.mark.parametrize("types", TYPES, ids=["f32", "bf16", "bf16-f32"])
@pytest.mark.parametrize("rows,dim", SIZES)
def test_forward_and_quant(ops, rows, dim, types):
    io, rt = types
    x, res = U.rand(1, rows, dim, dtype=io), U.rand(2, rows, dim, dtype=rt, scale=3.0)
    w = 1.0 + 0.2 * U.rand(3, dim)
    y, gy = U.guarded((rows, dim), io)
    r, gr = U.guarded((rows, dim), rt)
    ops.add_rms_norm(x, w, res, out=y, residual_out=r)
    q, gq = U.guarded((rows, dim), torch.float8_e4m3fn)
    sc, gs = U.guarded((rows,), F32)
    _, _, r2 = ops.add_rms_norm_quant(x, w, res, out=q, scale_out=sc)
    torch.cuda.synchronize()
    for g in (gy, gr, gq, gs):
        g()
    ro, yo, by = R.add_rms_norm(U.f64(x), U.f64(w), U.f64(res), bounds=True)
    U.close(r, ro, R.U * np.abs(ro), "r")
    assert torch.equal(r, r2)
    U.close(y, yo, by, "y")
    check_quant(q, sc, yo, by)


@pytest.mark.parametrize("types", TYPES, ids=["f32", "bf16", "bf16-f32"])
@pytest.mark.parametrize("rows,dim", SIZES + [(1000, 96), (700, 40), (4100, 768)])
def test_backward(ops, rows, dim, types):
    io, rt = types
    dy, r, dr = U.rand(4, rows, dim, dtype=io), U.rand(5, rows, dim, dtype=rt, scale=2.0), U.rand(6, rows, dim, dtype=rt)
    w = 1.0 + 0.2 * U.rand(7, dim)
    for add in (dr, None):
        got = ops.add_rms_norm_bwd(dy, r, w, dresidual=add)
        dro, dwo, bdr, bdw = R.add_rms_norm_bwd(U.f64(dy), U.f64(r), U.f64(w), U.f64(add), bounds=True)
        U.close(got["dx"], dro, bdr, "dx")
        U.close(got["dresidual"], dro, bdr, "dresidual")
        U.close(got["dweight"], dwo, bdw, "dweight")
        assert (got["dresidual"] is got["dx"]) == (io == rt)


# every split of a row over lanes and waves, with more rows than one round of workgroups where that is cheap
SPLITS = [(4200, 257), (30, 601), (2100, 1023), (40, 1999), (530, 2561), (9, 4001), (530, 6001), (30, 1280), (2100, 1500),
          (600, 2048), (530, 5120), (9, 12004), (9000, 120), (5000, 250)]


@pytest.mark.parametrize("types", TYPES, ids=["f32", "bf16", "bf16-f32"])
@pytest.mark.parametrize("rows,dim", SPLITS)
def test_rows_of_every_split(ops, rows, dim, types):
    io, rt = types
    x, r, w = U.rand(1, rows, dim, dtype=io), U.rand(2, rows, dim, dtype=rt, scale=2.0), 1.0 + 0.2 * U.rand(3, dim)
    y, _ = ops.add_rms_norm(x, w, r)
    q, sc, _ = ops.add_rms_norm_quant(x, w, r)
    _, yo, by = R.add_rms_norm(U.f64(x), U.f64(w), U.f64(r), bounds=True)
    U.close(y, yo, by, "y")
    check_quant(q, sc, yo, by)
    got = ops.add_rms_norm_bwd(x, r, w, dresidual=r)
    dro, dwo, bdr, bdw = R.add_rms_norm_bwd(U.f64(x), U.f64(r), U.f64(w), U.f64(r), bounds=True)
    U.close(got["dx"], dro, bdr, "dx")
    U.close(got["dresidual"], dro, bdr, "dresidual")
    U.close(got["dweight"], dwo, bdw, "dweight")


def test_without_a_residual(ops):
    x, w = U.rand(1, 6, 200, dtype=BF16), 1.0 + 0.1 * U.rand(2, 200)
    y, r = ops.add_rms_norm(x, w)
    assert r is None
    _, yo, by = R.add_rms_norm(U.f64(x), U.f64(w), bounds=True)
    U.close(y, yo, by)
    y2, r2 = ops.add_rms_norm(x, w, residual_dtype=F32)           # the residual stream starts here, in fp32
    assert torch.equal(y2, y) and torch.equal(r2, x.float())
    q, s, r3 = ops.add_rms_norm_quant(x, w)
    assert r3 is None
    check_quant(q, s, yo, by)


def test_the_residual_in_place(ops):
    for io, rt in TYPES:
        for dim in (768, 77):
            x, res, w = U.rand(1, 40, dim, dtype=io), U.rand(2, 40, dim, dtype=rt), 1.0 + 0.1 * U.rand(3, dim)
            y, r = ops.add_rms_norm(x, w, res)
            own = res.clone()
            y2, r2 = ops.add_rms_norm(x, w, own, residual_out=own)
            assert r2 is own and torch.equal(own, r) and torch.equal(y, y2)
            dy, dr = U.rand(4, 40, dim, dtype=io), U.rand(5, 40, dim, dtype=rt)
            want = ops.add_rms_norm_bwd(dy, r, w, dresidual=dr)
            got = ops.add_rms_norm_bwd(dy, r, w, dresidual=dr, dresidual_out=dr)
            assert got["dresidual"] is dr and torch.equal(dr, want["dresidual"]) and torch.equal(got["dx"], want["dx"])


@pytest.mark.parametrize("io", [F32, BF16])
def test_strided_and_unaligned_rows(ops, io):
    for dim, off, width in ((256, 256, 768), (256, 1, 300), (65, 3, 140)):
        wide = U.rand(1, 2, 9, width, dtype=io)
        x = wide[..., off:off + dim]
        res, w = U.rand(2, 2, 9, dim, dtype=io), 1.0 + 0.1 * U.rand(3, dim)
        y, r = ops.add_rms_norm(x, w, res)
        y2, r2 = ops.add_rms_norm(x.contiguous(), w, res)
        _, yo, by = R.add_rms_norm(U.f64(x), U.f64(w), U.f64(res), bounds=True)
        U.close(y, yo, by)
        U.close(y2, yo, by)
        assert torch.equal(r, r2)
        # the other tensors off their alignment as well
        buf = U.rand(4, 18 * dim + 1, dtype=io)[1:].view(2, 9, dim)
        U.close(ops.add_rms_norm(buf, w, res)[0], *R.add_rms_norm(U.f64(buf), U.f64(w), U.f64(res), bounds=True)[1:])
        got = ops.add_rms_norm_bwd(buf, res, w)
        dro, dwo, bdr, bdw = R.add_rms_norm_bwd(U.f64(buf).reshape(18, dim), U.f64(res).reshape(18, dim), U.f64(w), bounds=True)
        U.close(got["dx"].view(18, dim), dro, bdr)
        U.close(got["dweight"], dwo, bdw)


def test_rows_that_share_a_wave_with_eps_zero(ops):
    """The rows past the last one count for nothing, even where eps = 0 makes an absent row's scale infinite."""
    dy, r, w = U.rand(1, 13, 64, dtype=BF16), U.rand(2, 13, 64, dtype=BF16), 1.0 + 0.1 * U.rand(3, 64)
    got = ops.add_rms_norm_bwd(dy, r, w, eps=0.0)
    dro, dwo, bdr, bdw = R.add_rms_norm_bwd(U.f64(dy), U.f64(r), U.f64(w), eps=0.0, bounds=True)
    U.close(got["dx"], dro, bdr)
    U.close(got["dweight"], dwo, bdw)


def test_zero_tiny_huge_and_nan_rows(ops):
    x = U.rand(1, 8, 96)
    x[0] = 0.0
    x[1] *= 1e-30
    x[2] *= 1e15
    x[3, 5] = float("nan")
    x[4, 5] = float("inf")
    w = 1.0 + 0.1 * U.rand(2, 96)
    w1 = w.clone()
    w1[7] = 1e-42
    y, _ = ops.add_rms_norm(x, w)
    q, s, _ = ops.add_rms_norm_quant(x, w)
    assert not bool(y[0].any()) and not bool(q[0].float().any()) and float(s[0]) == 2.0 ** -126
    for i in (1, 2, 5, 6, 7):
        _, yo, by = R.add_rms_norm(U.f64(x[i:i + 1]), U.f64(w), bounds=True)
        U.close(y[i:i + 1], yo, by)
        check_quant(q[i:i + 1], s[i:i + 1], yo, by)
    assert bool(torch.isnan(y[3]).all()) and bool(torch.isnan(q[3].float()).all()) and bool(torch.isnan(s[3]))
    # an infinity: its square makes the row's rms infinite, every other value 0
    assert bool(torch.isnan(y[4, 5])) and not bool(y[4, :5].any()) and bool(torch.isnan(s[4]))
    tiny = ops.add_rms_norm_quant(x[5:6], torch.full_like(w, 1e-40))
    assert float(tiny[1]) == 2.0 ** -126 and bool(torch.isfinite(tiny[0].float()).all())


def test_weight_gradient_over_many_rows_repeats_to_the_bit(ops):
    dy, r, w = U.rand(1, 20000, 130, dtype=BF16), U.rand(2, 20000, 130, dtype=BF16), 1.0 + 0.1 * U.rand(3, 130)
    a, b = ops.add_rms_norm_bwd(dy, r, w), ops.add_rms_norm_bwd(dy, r, w)
    assert all(torch.equal(a[k], b[k]) for k in a)
    _, dwo, _, bdw = R.add_rms_norm_bwd(U.f64(dy), U.f64(r), U.f64(w), bounds=True)
    U.close(a["dweight"], dwo, bdw)


def test_no_rows(ops):
    x, w = torch.empty(0, 64, device="cuda"), torch.ones(64, device="cuda")
    assert ops.add_rms_norm(x, w)[0].shape == (0, 64)
    assert not bool(ops.add_rms_norm_bwd(x, x, w)["dweight"].any())


def test_leading_axes(ops):
    """One row without leading axes, and three leading axes: the same rows."""
    w = 1.0 + 0.1 * U.rand(2, 96)
    x, res = U.rand(1, 2, 3, 5, 96, dtype=BF16), U.rand(3, 2, 3, 5, 96)
    y, r = ops.add_rms_norm(x, w, res)
    q, s, _ = ops.add_rms_norm_quant(x, w, res)
    g = ops.add_rms_norm_bwd(x, res, w)
    assert s.shape == (2, 3, 5)
    i = (1, 2, 3)
    y1, r1 = ops.add_rms_norm(x[i], w, res[i])
    q1, s1, _ = ops.add_rms_norm_quant(x[i], w, res[i])
    assert s1.shape == () and torch.equal(y1, y[i]) and torch.equal(r1, r[i]) and torch.equal(s1, s[i])
    assert torch.equal(q1.view(torch.uint8), q[i].view(torch.uint8))
    assert torch.equal(ops.add_rms_norm_bwd(x[i], res[i], w)["dx"], g["dx"][i])


def test_on_another_stream(ops):
    x, w, res = U.rand(1, 4000, 768, dtype=BF16), 1.0 + 0.1 * U.rand(2, 768), U.rand(3, 4000, 768)
    want = ops.add_rms_norm(x, w, res)[0], ops.add_rms_norm_bwd(x, res, w)["dweight"]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = ops.add_rms_norm(x, w, res)[0], ops.add_rms_norm_bwd(x, res, w)["dweight"]
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_graph_replays(ops):
    from test_gpu_graph import replay_matches_eager
    t = dict(x=U.rand(1, 300, 768, dtype=BF16), res=U.rand(2, 300, 768), w=1.0 + 0.1 * U.rand(3, 768),
             dy=U.rand(4, 300, 768, dtype=BF16))

    def fn(t):
        y, r = ops.add_rms_norm(t["x"], t["w"], t["res"])
        q, s, _ = ops.add_rms_norm_quant(t["x"], t["w"], t["res"])
        g = ops.add_rms_norm_bwd(t["dy"], r, t["w"], dresidual=t["res"])
        return [y, r, q.view(torch.uint8), s] + list(g.values())

    def refill(t, r):
        for k in ("x", "res", "dy"):
            t[k].copy_(torch.randn(t[k].shape, device="cuda"))
    replay_matches_eager(t, fn, refill)


def test_offsets_past_32_bits(ops):
    rows, dim = 300000, 8192                                       # 4.9 GB of bf16
    x = torch.empty(rows, dim, dtype=BF16, device="cuda").normal_()
    w = 1.0 + 0.1 * U.rand(3, dim)
    y, _ = ops.add_rms_norm(x, w)
    assert torch.equal(y[-7:], ops.add_rms_norm(x[-7:], w)[0])
    q, s, _ = ops.add_rms_norm_quant(x, w)
    q7, s7, _ = ops.add_rms_norm_quant(x[-7:], w)
    assert torch.equal(q[-7:].view(torch.uint8), q7.view(torch.uint8)) and torch.equal(s[-7:], s7)
    got = ops.add_rms_norm_bwd(y, x, w)
    assert torch.equal(got["dx"][-7:], ops.add_rms_norm_bwd(y[-7:], x[-7:], w)["dx"])


def test_refusals(ops):
    x, w = U.rand(1, 4, 64, dtype=BF16), torch.ones(64, device="cuda")
    for bad in (lambda: ops.add_rms_norm(x.half(), w), lambda: ops.add_rms_norm(x, w.bfloat16()),
                lambda: ops.add_rms_norm(x, w[:32]), lambda: ops.add_rms_norm(x, w, x[:2]),
                lambda: ops.add_rms_norm(x.float(), w, x), lambda: ops.add_rms_norm(x, w, x.half()),
                lambda: ops.add_rms_norm(x, w, x, residual_dtype=F32), lambda: ops.add_rms_norm(x, w, eps=-1.0),
                lambda: ops.add_rms_norm(x.cpu(), w), lambda: ops.add_rms_norm(x.t(), w[:4]),
                lambda: ops.add_rms_norm_bwd(x, x[:2], w), lambda: ops.add_rms_norm_bwd(x.float(), x, w),
                lambda: ops.add_rms_norm(torch.empty(2, 32769, device="cuda"), torch.empty(32769, device="cuda"))):
        with pytest.raises((ValueError, RuntimeError)):
            bad()
    with pytest.raises(RuntimeError, match="ALIAS"):
        ops.add_rms_norm(x, w, out=x)



def near_middles(dim, power=0):
    """dim weights, the largest 1.7 * 2^power, whose quotients by the row's scale, a 448th of it in fp32, lie on or one
    ulp beside the middle of two e4m3 numbers; the scale; and the e4m3 numbers of the fp32 quotients."""
    top = np.ldexp(np.float32(1.7), power)
    scale = np.maximum(top / np.float32(448.0), np.float32(2.0 ** -126))
    e4m3 = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()    # 0 .. 448
    middle = ((e4m3[1:] + e4m3[:-1]) / 2)[np.arange(dim) * 37 % 126]
    w = np.minimum((middle * float(scale)).astype(np.float32), top)
    beside = np.arange(dim) % 3
    w = np.where(beside == 1, np.nextafter(w, np.float32(0)), np.where(beside == 2, np.nextafter(w, top), w))
    w[dim // 2] = top
    to8 = lambda v: torch.from_numpy(v).to(torch.float8_e4m3fn)
    return w, scale, to8(w / scale), to8(w * (np.float32(1) / scale))


def test_a_product_with_the_reciprocal_is_told_from_the_quotient():
    _, _, q, by_reciprocal = near_middles(2048)
    assert int((q.view(torch.uint8) != by_reciprocal.view(torch.uint8)).sum()) > 20


@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("dim", [64, 256, 2048, 4096, 8192, 32768])
@pytest.mark.parametrize("types", TYPES, ids=["f32", "bf16", "bf16-f32"])
def test_the_8_bit_output_is_the_rounded_quotient(ops, types, dim, off):
    """Rows of +-3 with eps = 0: the mean square is 9, its root 3 and r / 3 exactly +-1 in fp32, so y is the weight
    (taken in the formula's order) and q = e4m3(y / scale) can be said to the bit, down to the smallest scales."""
    io, rt = types
    sign = torch.where(U.rand(1, 9, dim) < 0, -1.0, 1.0)
    x = torch.zeros(9 * dim + off, dtype=io, device="cuda")[off:].view(9, dim).copy_(sign * 2)
    res = torch.zeros(9 * dim + off, dtype=rt, device="cuda")[off:].view(9, dim).copy_(sign)
    for power in (0, 90, -80, -84, -110, -117, -119):
        w, scale, want, _ = near_middles(dim, power)
        wt = torch.zeros(dim + off, device="cuda")[off:].copy_(torch.from_numpy(w))
        q, s, _ = ops.add_rms_norm_quant(x, wt, res, eps=0.0)
        assert bool((s.cpu() == float(scale)).all()), power
        assert torch.equal(q.float().cpu(), want.float() * sign.cpu()), power
    w, _, _, _ = near_middles(dim)
    wt = torch.zeros(dim + off, device="cuda")[off:].copy_(torch.from_numpy(w))
    assert torch.equal(ops.add_rms_norm(x, wt, res, eps=0.0)[0], (wt * sign).to(io))


def test_an_output_past_fp32_has_an_infinite_scale(ops):
    """The finite values of such a row are 0 in 8 bits, the infinite ones NaN; other rows have none of it."""
    x = torch.ones(3, 64, device="cuda")
    x[1, :8] = 8.0
    w = torch.full((64,), 2e38, device="cuda")
    q, s, _ = ops.add_rms_norm_quant(x, w)
    y, _ = ops.add_rms_norm(x, w)
    assert bool(torch.isinf(y[1, :8]).all()) and bool(torch.isfinite(y[1, 8:]).all()) and bool(torch.isinf(s[1]))
    assert bool(torch.isnan(q[1, :8].float()).all()) and not bool(q[1, 8:].float().any())
    assert bool((q[[0, 2]].float() == 448.0).all())


@pytest.mark.parametrize("types", TYPES, ids=["f32", "bf16", "bf16-f32"])
@pytest.mark.parametrize("rows,dim,ld,off", [(13, 64, 192, 64), (13, 64, 65, 1), (7, 1, 3, 2), (37, 24, 32, 8), (9, 100, 301, 0),
                                             (4100, 768, 1536, 768), (33, 2561, 2600, 3), (5, 4096, 8192, 4096),
                                             (3, 12001, 12005, 4), (2, 64, (1 << 24) + 64, 0), (1, 130, 500, 370)])
def test_gradient_at_a_strided_row(ops, types, rows, dim, ld, off):
    """The r of a forward without residual is x itself, rows apart as they may be."""
    io, rt = types
    wide = torch.empty(rows, ld, dtype=rt, device="cuda")
    x = wide[:, off:off + dim]
    x.copy_(U.rand(1, rows, dim))
    wide[:, off + dim:] = float("nan")                             # what lies between the rows counts for nothing
    wide[:, :off] = float("nan")
    dy, dr, w = U.rand(2, rows, dim, dtype=io), U.rand(3, rows, dim, dtype=rt), 1.0 + 0.2 * U.rand(4, dim)
    if io == rt:
        assert ops.add_rms_norm(x, w)[1] is None
    for add in (None, dr):
        got, want = ops.add_rms_norm_bwd(dy, x, w, dresidual=add), ops.add_rms_norm_bwd(dy, x.contiguous(), w, dresidual=add)
        dro, dwo, bdr, bdw = R.add_rms_norm_bwd(U.f64(dy), U.f64(x), U.f64(w), U.f64(add), bounds=True)
        for g in (got, want):
            U.close(g["dx"], dro, bdr, "dx")
            U.close(g["dresidual"], dro, bdr, "dresidual")
            U.close(g["dweight"], dwo, bdw, "dweight")
            assert g["dresidual"].is_contiguous()


def test_gradient_at_strided_rows_past_32_bits(ops):
    rows, dim, ld = 300000, 64, 8192                               # 4.9 GB of bf16 between the first row and the last
    wide = torch.empty(rows, ld, dtype=BF16, device="cuda")
    x = wide[:, 128:128 + dim].normal_()
    dy, w = U.rand(2, rows, dim, dtype=BF16), 1.0 + 0.1 * U.rand(3, dim)
    got, want = ops.add_rms_norm_bwd(dy, x, w), ops.add_rms_norm_bwd(dy, x.contiguous(), w)
    assert torch.equal(got["dx"], want["dx"]) and torch.equal(got["dweight"], want["dweight"])


def test_gradient_refuses_overlapping_and_uneven_rows(ops):
    x, w = U.rand(1, 4, 6, 64), torch.ones(64, device="cuda")
    dy = x[:, :3].contiguous()
    with pytest.raises(ValueError, match="evenly"):
        ops.add_rms_norm_bwd(dy, x[:, :3], w)
    with pytest.raises(ValueError, match="overlap"):
        ops.add_rms_norm_bwd(dy, x[:1, :1].expand(4, 3, 64), w)
    with pytest.raises(ValueError):
        ops.add_rms_norm_bwd(dy, x[:, :3].transpose(0, 1).contiguous(), w)
