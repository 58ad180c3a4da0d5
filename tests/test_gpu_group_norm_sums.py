"""The group norm's sums where they are long, far from zero, or over many batch entries."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_util as U
import test_gpu_group_norm as G

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


# entries whose groups stay in registers, and that are cut into runs of rows
@pytest.mark.parametrize("R", [2, 20, 64, 1500, 3000])
@pytest.mark.parametrize("C,groups", [(64, 4), (30, 2), (2100, 2)])
def test_groups_far_from_zero_with_next_to_no_spread(ops, R, C, groups):
    """Values whose mean is a fp32 number, so that (x - mean) is exact and the statistics are good to their own
    roundings: the sums' 10 U, and 8 U for the square root and the quotient."""
    x = torch.full((2, R, C), 100004.0, device="cuda")
    D = C // groups
    x[0, ::2, :D] += 2.0 ** -6                                             # x = c, c + 2^-6 in turn: variance 2^-14
    x[1, :, D:] = 16777213.0                                               # 24 bits long
    b = U.rand(1, C)
    y, mean, rstd = ops.group_norm(x, groups, bias=b, eps=1e-5, return_stats=True)
    m, v = np.full((2, groups), 100004.0), np.zeros((2, groups))
    m[0, 0], v[0, 0] = 100004.0 + 2.0 ** -7, 2.0 ** -14
    m[1, 1:] = 16777213.0
    assert np.array_equal(U.f64(mean), m)
    want = 1.0 / np.sqrt(v + float(np.float32(1e-5)))
    assert (np.abs(U.f64(rstd) - want) <= 18 * EPS * want).all()
    rep = lambda t: np.repeat(t, D, axis=-1)[:, None]
    yo = (U.f64(x) - rep(m)) * rep(want) + U.f64(b)
    U.close(y, yo, 30 * EPS * (np.abs(yo) + np.abs(U.f64(b))), "y")


# batch entries that share workgroups in the gradient: one wide row, few rows, rows beyond a workgroup's registers
FOLDED = [(1500, 1, 4104, 1), (1100, 1, 5000, 2), (3000, 4, 40, 40), (2500, 2, 256, 4), (600, 64, 264, 1), (1030, 65, 130, 2),
          (40000, 2, 24, 3)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,R,C,groups", FOLDED)
def test_many_entries(ops, N, R, C, groups, dtype):
    G.check(ops, G.inputs(N, R, C, DT[dtype], gate=R % 2 == 0, affine=True, seed=R), groups, silu=R != 2)


def one_signed(ops, N, R, D, groups):
    """dy = 1 and x = 1/2 throughout, with mean 0 and rstd 1: da is SiLU's slope at weight / 2 + bias, the same in all
    rows, and its sums are N R of it.  At most 128 values are added in fp32 before a sum moves on, 128 such sums after
    it, some threads' and waves' sums and one more rounding of each: 300 U; the slope itself is off by
    (2 |a| + 40) U relative to 1.1, its largest value."""
    C = D * groups
    shape = (N, R, C) if R > 1 else (N, C)
    x = torch.full(shape, 0.5, dtype=torch.bfloat16, device="cuda")
    dy = torch.ones(shape, dtype=torch.bfloat16, device="cuda")
    w, b = U.rand(1, C), U.rand(2, C)
    got = ops.group_norm_bwd(dy, x, torch.zeros(N, groups, device="cuda"), torch.ones(N, groups, device="cuda"), groups, w, b,
                             activation="silu")
    a = 0.5 * U.f64(w) + U.f64(b)
    s = 1.0 / (1.0 + np.exp(-a))
    da = s * (1.0 + a * (1.0 - s))
    allowed = N * R * EPS * (300.0 * np.abs(da) + 1.1 * (2.0 * np.abs(a) + 40.0))
    for name, f in (("dbias", 1.0), ("dweight", 0.5)):
        over = np.abs(U.f64(got[name]) - f * N * R * da) / (f * allowed)
        assert over.max() <= 1.0, f"{name}: {over.max():.3g} times what is allowed"


def test_one_signed_gradients_over_many_rows(ops):
    """More workgroups than the GPU holds before any entry is cut: 4096 rows to a thread."""
    one_signed(ops, 17, 8192, 255, 64)


def test_one_signed_gradients_over_many_tokens(ops):
    """Groups that fill the GPU by themselves: 4096 tokens to a wave."""
    one_signed(ops, 16384, 1, 2, 16384)


def test_more_entries_than_a_launch_has_rows_of(ops):
    """Entries too long to share workgroups, more than a launch's second axis holds."""
    G.check(ops, G.inputs(66000, 65, 1, torch.float32, seed=7), 1)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("R,C", [(3000, 64), (2, 4100)])
def test_a_bad_first_value_stays_in_its_group(ops, R, C, bad):
    """The first value of a group is what its runs' sums are joined about."""
    D = C // 4
    t = G.inputs(3, R, C, torch.float32, seed=5)
    clean = ops.group_norm(t["x"], 4, t["weight"], t["bias"])
    t["x"][1, 0, D] = bad
    y, mean, rstd = ops.group_norm(t["x"], 4, t["weight"], t["bias"], return_stats=True)
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[1, :, D:2 * D] = True
    assert bool(torch.isnan(y[1, 0, D])) and torch.equal(y[~hit], clean[~hit])
    assert int(torch.isfinite(mean).sum()) == 11 and not bool(torch.isfinite(rstd[1, 1]))
