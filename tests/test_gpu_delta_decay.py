"""The gated delta rule's decays over their whole range, element by element.

With beta = 0 a state is h0 times the decays alone, so every element of it is known to a relative error:

    fp32 io, and the decode token: the exponential of a 64-bit sum is good to 4 U (its reduced argument, the series'
    steps and the last rounding); applying it is one rounding more.
    bf16 io: the exponential is the hardware's, good to 2 U, of an argument rounded to fp32: |G| / 2 U more.

(U = 2^-24.)  A product with q or with dy adds fp32 roundings, one per term at most, and in bf16 io 2^-17 of each term for
the two terms that computed operands have; a decay's result below fp32's smallest normal number counts as that."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_util as U

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS, TINY = 2.0 ** -24, 2.0 ** -126


@pytest.fixture(scope="module", autouse=True)
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from selective_scan_ssm_amd import _lib, ops
    _lib.load()
    return ops


def within(got, want, allowed, name):
    g = U.f64(got)
    assert g.shape == want.shape and np.isfinite(g).all(), name
    over = np.abs(g - want) / allowed
    i = np.unravel_index(np.argmax(over), g.shape)
    assert over[i] <= 1.0, f"{name}: {g[i]} for {want[i]} at {i}, {over[i]:.3g} times what is allowed"


def unit(seed, *shape, dtype):
    t = U.rand(seed, *shape)
    return (t / t.norm(dim=-1, keepdim=True)).to(dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [24, 64, 128])
def test_one_token_only_decays(ops, K, dtype):
    """g from near 0 to beyond fp32's range, a head to each."""
    H, V, io = 100, 40, DT[dtype]
    g = -torch.arange(H, device="cuda").float() * 1.07 - 0.01
    q, k, v = unit(1, 2, H, K, dtype=io), unit(2, 2, H, K, dtype=io), U.rand(3, 2, H, V, dtype=io)
    before = U.rand(4, 2, H, V, K)
    state = before.clone()
    y = ops.delta_state_update(state, q, k, v, g.expand(2, H).contiguous(), torch.zeros(2, H, device="cuda"), scale=0.3)
    s, a = U.f64(before), np.exp(U.f64(g))[None, :, None, None]
    within(state, a * s, 6 * EPS * a * np.abs(s) + TINY, "state")
    sq = np.einsum("bhvk,bhk->bhv", s, U.f64(q))
    terms = np.einsum("bhvk,bhk->bhv", np.abs(s), np.abs(U.f64(q)))
    want = 0.3 * a[..., 0] * sq
    # a lane's four terms and up to five folds, the exponential, three products
    within(y, want, 18 * EPS * 0.3 * a[..., 0] * terms + U.HALF_STEP[io] * np.abs(want) + TINY, "y")


# a head to each: memories of one to some hundred steps, decays whose steps alone leave fp32's accuracy near 1
RATES = [0.003, 0.02, 0.11, 0.25, 0.5, 0.77, 1.3, 3.1, 8.3, 15.7, 16.9, 29.0, 59.0, 86.0]


def exponential(dtype, G):
    """The relative error of exp(G) and of applying it, in U."""
    return 5.0 + (0.0 if dtype == "f32" else 0.5) * np.abs(G)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,K", [(64, 64), (150, 32), (70, 128)])
def test_a_sequence_only_decays(ops, T, K, dtype):
    H, V, io = len(RATES), 24, DT[dtype]
    chunks = -(-T // 64)
    g = -torch.tensor(RATES, device="cuda").expand(1, T, H).contiguous()
    q, k, v = unit(1, 1, T, H, K, dtype=io), unit(2, 1, T, H, K, dtype=io), U.rand(3, 1, T, H, V, dtype=io)
    beta, h0 = torch.zeros(1, T, H, device="cuda"), U.rand(4, 1, H, V, K)
    y, last = ops.delta_scan_fwd(q, k, v, g, beta, scale=0.3, h0=h0, return_last_state=True)
    dy, dl = U.rand(5, 1, T, H, V, dtype=io), U.rand(6, 1, H, V, K)
    got = ops.delta_scan_bwd(q, k, v, g, beta, torch.zeros_like(dy), scale=0.3, h0=h0, dlast=dl)
    dq = ops.delta_scan_bwd(q, k, v, g, beta, dy, scale=0.3, h0=h0)["dq"]
    G = np.cumsum(U.f64(g), 1)                                             # (1, T, H)
    a, s, q64, dy64 = np.exp(G), U.f64(h0), U.f64(q), U.f64(dy)
    end = a[:, -1, :, None, None]
    rel = chunks * EPS * exponential(dtype, G[:, -1])[..., None, None]
    within(last, end * s, rel * end * np.abs(s) + TINY, "last")
    within(got["dh0"], end * U.f64(dl), rel * end * np.abs(U.f64(dl)) + TINY, "dh0")
    two = 0.0 if dtype == "f32" else 2.0 ** -17
    half = U.HALF_STEP[io]
    for name, t, want, terms, n in (
            ("y", y, np.einsum("bhvk,bthk->bthv", s, q64), np.einsum("bhvk,bthk->bthv", np.abs(s), np.abs(q64)), K),
            ("dq", dq, np.einsum("bhvk,bthv->bthk", s, dy64), np.einsum("bhvk,bthv->bthk", np.abs(s), np.abs(dy64)), V)):
        d = 0.3 * a[..., None]
        each = (chunks * exponential(dtype, G) + n + 4)[..., None] * EPS + two
        within(t, d * want, each * d * terms + half * np.abs(d * want) + n * TINY, name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_cut_sequence_only_decays(ops, dtype):
    """Long enough to be cut in time: the segments' transitions are decays of up to some hundred steps."""
    T, K, V, io = 3000, 64, 24, DT[dtype]
    rates = [0.0004, 0.004, 0.012, 0.027]
    H = len(rates)
    g = -torch.tensor(rates, device="cuda").expand(1, T, H).contiguous()
    q, v = unit(1, 1, T, H, K, dtype=io), U.rand(3, 1, T, H, V, dtype=io)
    beta, h0 = torch.zeros(1, T, H, device="cuda"), U.rand(4, 1, H, V, K)
    dl = U.rand(6, 1, H, V, K)
    _, last = ops.delta_scan_fwd(q, q, v, g, beta, h0=h0, return_last_state=True)
    dh0 = ops.delta_scan_bwd(q, q, v, g, beta, torch.zeros_like(v), h0=h0, dlast=dl)["dh0"]
    G = T * U.f64(g)[:, 0]
    # at most 47 segments of a chunk each, at each of which the state goes through a product with one term that is not 0
    each = 47 * (exponential(dtype, G / 47) * EPS + (2 * EPS if dtype == "f32" else 3 * 2.0 ** -17))[..., None, None]
    a = np.exp(G)[..., None, None]
    for name, t, s in (("last", last, U.f64(h0)), ("dh0", dh0, U.f64(dl))):
        within(t, a * s, each * a * np.abs(s) + TINY, name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("restart", [float("-inf"), -104.0, -90.0])
def test_steps_behind_many_restarts(ops, restart, dtype):
    """A state written behind many restarts (padding on the left) decays as if they had not been there."""
    K, V, H, T, io = 32, 24, 6, 64, DT[dtype]
    n = 47                                                                 # the last restart
    g = -(U.rand(9, 1, T, H).abs() * 0.1 + 0.003)
    g[:, :n + 1] = restart
    beta = torch.zeros(1, T, H, device="cuda")
    beta[:, n] = 1.0
    k = torch.zeros(1, T, H, K, device="cuda")
    k[..., 3] = 1.0
    v = U.rand(3, 1, T, H, V, dtype=io)
    y, last = ops.delta_scan_fwd(k.to(io), k.to(io), v, g, beta, scale=0.5, return_last_state=True)
    dl = U.rand(6, 1, H, V, K)
    got = ops.delta_scan_bwd(k.to(io), k.to(io), v, g, beta, torch.zeros_like(v), scale=0.5, dlast=dl)
    G = np.concatenate([np.zeros((1, 1, H)), np.cumsum(U.f64(g)[:, n + 1:], 1)], 1)
    a, vn = np.exp(G), U.f64(v)[:, n]                                      # (1, T - n, H), (1, H, V)
    want = np.zeros((1, H, V, K))
    want[..., 3] = a[:, -1, :, None] * vn
    # U and U exp(G_end - G) are computed operands (two bf16 terms), the decay is rounded twice
    rel = 8 * EPS + (0.0 if dtype == "f32" else 2.0 ** -17)
    within(last, want, rel * np.abs(want) + TINY, "last")
    wy = 0.5 * a[..., None] * vn[:, None]
    within(y[:, n:], wy, (2 * rel + U.HALF_STEP[io]) * np.abs(wy) + TINY, "y")
    # dbeta = <dlast, last>, dg of the steps behind the same: V products that are operands on both sides
    dot, terms = ((U.f64(dl) * t).sum((-1, -2)) for t in (want, np.abs(np.sign(U.f64(dl)) * want)))
    allowed = (3 * rel + (V + 64) * EPS) * terms + TINY
    within(got["dbeta"][:, n], dot, allowed, "dbeta")
    for t in range(n + 1, T):
        within(got["dg"][:, t], dot, allowed, f"dg at {t}")


def test_no_key_channels_are_refused_as_a_shape(ops):
    q, v, g = torch.zeros(1, 4, 2, 0, device="cuda"), torch.zeros(1, 4, 2, 8, device="cuda"), torch.zeros(1, 4, 2, device="cuda")
    with pytest.raises(RuntimeError, match="invalid arguments|SHAPE"):
        ops.delta_scan_fwd(q, q, v, g, g)
    with pytest.raises(RuntimeError, match="SHAPE"):
        ops.delta_state_update(torch.zeros(1, 2, 8, 0, device="cuda"), q[:, 0], q[:, 0], v[:, 0], g[:, 0], g[:, 0])
