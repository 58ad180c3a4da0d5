"""The global gradient norm and clipping on the GPU against their fp64 definition."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_util as U
from oracle import recurrent_block as R

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from selective_scan_ssm_amd import _lib, ops
    _lib.load()
    return ops


def grads(sizes, kinds=(F32, BF16), seed=0, scale=1.0):
    return [U.rand(seed + i, *((n,) if isinstance(n, int) else n), dtype=kinds[i % len(kinds)], scale=scale)
            for i, n in enumerate(sizes)]


def norm_close(norm, want):
    # the 64-bit sum is rounded to fp32 once after the root
    assert abs(float(norm) - want) <= 2 * R.U * want, (float(norm), want)


# one tensor; many tiny ones; ends around the runs of 4096; more tensors than one table holds; large ones
LISTS = [[1], [3] * 1000, [1024, 1023, 1025, 2048, 2049, 4096, 5000], [100] * 119 + [5000], [70] * 120, [70] * 121,
         [5, 1, 7], [16383, 16384, 16385, 3], [(33, 65), 1, 100000, 0, 17], [8] * 300, [1000003, 70001]]


@pytest.mark.parametrize("kinds", [(F32,), (BF16,), (F32, BF16)], ids=["f32", "bf16", "mixed"])
@pytest.mark.parametrize("sizes", LISTS, ids=lambda s: f"{len(s)}x{s[0]}")
def test_norm_and_clip(ops, sizes, kinds):
    g = grads(sizes, kinds)
    host = [U.f64(t) for t in g]
    want, coef = R.clip(host, 0.5)
    norm_close(ops.grad_norm(g), want)
    outs, checks = zip(*[U.guarded(t.shape, F32 if i % 3 else BF16) for i, t in enumerate(g)])
    keep = [t.clone() for t in g]
    norm_close(ops.clip_grads(g, 0.5, out=outs), want)
    for o, h, c, t, k in zip(outs, host, checks, g, keep):
        c()
        U.close(o, h * coef, np.abs(h * coef) * 6 * R.U, "out")
        assert torch.equal(t, k)
    norm_close(ops.clip_grads(g, 0.5), want)                       # in place
    for t, h in zip(g, host):
        U.close(t, h * coef, np.abs(h * coef) * 6 * R.U, "in place")


def test_below_the_limit_nothing_changes(ops):
    g = grads([4096, 33, 70000])
    keep = [t.clone() for t in g]
    want, _ = R.clip([U.f64(t) for t in g], 1.0)
    for limit in (want * 1.01, float("inf")):
        norm_close(ops.clip_grads(g, limit), want)
        assert all(torch.equal(a, b) for a, b in zip(g, keep))
    out = [torch.empty(t.shape, device="cuda") for t in g]
    ops.clip_grads(g, want * 2, out=out)
    assert all(torch.equal(o, t.float()) for o, t in zip(out, g))


def test_a_limit_of_zero_and_zero_gradients(ops):
    g = grads([100, 50])
    ops.clip_grads(g, 0.0)
    assert not any(bool(t.any()) for t in g)
    assert float(ops.clip_grads(g, 1.0)) == 0.0 and not any(bool(t.any()) for t in g)
    assert float(ops.clip_grads([torch.empty(0, device="cuda")], 1.0)) == 0.0


def test_unaligned_views_of_one_buffer(ops):
    for dt in (F32, BF16):
        buf = U.rand(3, 40000, dtype=dt)
        keep = buf.clone()
        cuts = [1, 4, 11, 12, 300, 1001, 20002, 39999]
        g = [buf[a:b] for a, b in zip(cuts, cuts[1:])]
        host = [U.f64(t) for t in g]
        want, coef = R.clip(host, 1.0)
        outbuf = torch.full((40008,), 7.0, device="cuda")
        out = [outbuf[a + 5:b + 5] for a, b in zip(cuts, cuts[1:])]
        norm_close(ops.clip_grads(g, 1.0, out=out), want)
        for o, h in zip(out, host):
            U.close(o, h * coef, np.abs(h * coef) * 6 * R.U)
        assert bool((outbuf[:6] == 7).all()) and bool((outbuf[40004:] == 7).all())
        norm_close(ops.clip_grads(g, 1.0), want)
        for t, h in zip(g, host):
            U.close(t, h * coef, np.abs(h * coef) * 6 * R.U)
        assert torch.equal(buf[:1], keep[:1]) and torch.equal(buf[39999:], keep[39999:])


def test_large_values_and_non_finite_ones(ops):
    big = [torch.full((1000,), 3e25, device="cuda"), torch.full((10,), 1e-30, device="cuda")]     # squares past fp32
    norm_close(ops.grad_norm(big), R.clip([U.f64(t) for t in big], 1.0)[0])
    for v in (float("inf"), float("nan")):
        g = grads([100, 50])
        g[1][3] = v
        n = float(ops.clip_grads(g, 1.0))
        assert n == v or n != n
        if v != v:
            assert all(bool(torch.isnan(t.float()).all()) for t in g)
        else:
            assert bool(torch.isnan(g[1][3])) and not bool(g[0].any())


def test_one_tensor_listed_twice(ops):
    g = grads([100])[0]
    want, _ = R.clip([U.f64(g), U.f64(g)], 1.0)
    norm_close(ops.grad_norm([g, g]), want)
    with pytest.raises(RuntimeError, match="ALIAS"):
        ops.clip_grads([g, g], 1.0)


def test_repeats_to_the_bit_and_replays(ops):
    from test_gpu_graph import replay_matches_eager
    t = {"g": grads([70000, 33, 8192, 1] * 40, scale=0.01)}
    out = [torch.empty(x.shape, device="cuda") for x in t["g"]]
    a = ops.clip_grads(t["g"], 0.1, out=out).clone()
    assert all(torch.equal(a, ops.clip_grads(t["g"], 0.1, out=out)) for _ in range(4))

    def fn(t):
        o = [torch.empty(x.shape, device="cuda") for x in t["g"]]
        n = ops.clip_grads(t["g"], 0.1, out=o)
        return [n, ops.grad_norm(t["g"])] + o

    def refill(t, r):
        for x in t["g"]:
            x.copy_(torch.randn(x.shape, device="cuda"))
    replay_matches_eager(t, fn, refill)


def test_more_than_four_billion_bytes(ops):
    g = torch.empty((1 << 31) + 12345, dtype=BF16, device="cuda").fill_(2.0 ** -16)
    assert abs(float(ops.grad_norm([g])) - 2.0 ** -16 * g.numel() ** 0.5) < 1e-6
    ops.clip_grads([g], 2.0 ** -17 * g.numel() ** 0.5, eps=0.0)
    assert bool((g[:5] == 2.0 ** -17).all()) and bool((g[-5:] == 2.0 ** -17).all())


def test_refusals(ops):
    g = grads([64, 32])
    for bad in (lambda: ops.clip_grads([], 1.0), lambda: ops.clip_grads([t.half() for t in g], 1.0),
                lambda: ops.clip_grads([t.cpu() for t in g], 1.0), lambda: ops.clip_grads([g[0][::2]], 1.0),
                lambda: ops.clip_grads(g, -1.0), lambda: ops.clip_grads(g, float("nan")), lambda: ops.clip_grads(g, None),
                lambda: ops.clip_grads(g, 1.0, out=[g[0]]), lambda: ops.clip_grads(g, 1.0, out=[g[1], g[0]]),
                lambda: ops.clip_grads(g, 1.0, norm_out=torch.empty(2, device="cuda")),
                lambda: ops.clip_grads([g[0], g[1].cpu()], 1.0)):
        with pytest.raises((ValueError, RuntimeError)):
            bad()


@pytest.mark.parametrize("limit", [1e38, 1.0])
def test_a_norm_past_fp32_still_scales(ops, limit):
    """Finite gradients whose norm fp32 does not hold: the norm is written as infinite, the coefficient is the formula's."""
    make = lambda: [torch.full((4000,), 3e38, device="cuda"), torch.full((33,), -2e38, device="cuda").to(BF16), U.rand(1, 7)]
    g = make()
    host = [U.f64(t) for t in g]
    norm, coef = R.clip(host, limit)
    assert norm > 3.5e38
    out = [torch.empty(t.shape, device="cuda") for t in g]
    assert float(ops.grad_norm(g)) == float("inf") and float(ops.clip_grads(g, limit, out=out)) == float("inf")
    own = make()
    ops.clip_grads(own, limit)
    for o, p, h in zip(out, own, host):
        # a coefficient below 2^-126 is held to 2^-150
        U.close(o, h * coef, np.abs(h) * (6 * R.U * coef + 2.0 ** -150))
        U.close(p, h * coef, np.abs(h) * (6 * R.U * coef + 2.0 ** -150))


def test_nothing_changes_at_or_below_the_limit_whatever_it_is(ops):
    """norm + eps <= max_norm, also where the quotient is 0 / 0 or inf / inf."""
    zero = [torch.zeros(100, device="cuda"), torch.zeros(9, dtype=BF16, device="cuda")]
    assert float(ops.clip_grads(zero, 0.0, eps=0.0)) == 0.0 and not any(bool(t.any()) or bool(t.isnan().any()) for t in zero)
    for first in (float("inf"), 3e38):
        g = [U.rand(1, 5000), U.rand(2, 70, dtype=BF16)]
        g[0][:40] = first
        keep = [t.clone() for t in g]
        assert float(ops.clip_grads(g, float("inf"))) == float("inf")
        assert all(torch.equal(a, b) for a, b in zip(g, keep))
    g[1][3] = float("nan")
    ops.clip_grads(g, float("inf"))
    assert all(bool(t.isnan().all()) for t in g)
