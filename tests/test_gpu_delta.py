"""The gated delta rule on the GPU against its step-by-step fp64 definition
(oracle/mixer.py), within the tolerance derived in mixer_util.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_util as U
import mixer_util as D
from oracle import mixer as M

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
NAMES = ("q", "k", "v", "g", "beta")


@pytest.fixture(scope="module", autouse=True)
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from selective_scan_ssm_amd import _lib, ops
    _lib.load()
    return ops


def args(t):
    return [t[n] for n in NAMES]


def check_fwd(ops, t, scale=0.3, want_ckpt=True):
    B, T, H, V = t["v"].shape
    K, io = t["q"].shape[-1], t["q"].dtype
    y, guard = U.guarded((B, T, H, V), io)
    last, lguard = U.guarded((B, H, V, K), torch.float32)
    ck = torch.full(ops.delta_ckpt_shape(t["q"], t["v"]), float("nan"), device="cuda") if want_ckpt else None
    ops.delta_scan_fwd(*args(t), scale=scale, h0=t["h0"], return_last_state=True, out=y, last_state_out=last, ckpt_out=ck)
    torch.cuda.synchronize()
    guard()
    lguard()
    yo, st = M.delta_rule(scale=scale, **D.host(t))
    D.close(y, yo, io, T, "y", size=scale * D.rms(st) * K ** 0.5 * D.rms(U.f64(t["q"])))
    D.close(last, st[-1], io, T, "last", size=D.rms(st))
    if want_ckpt and T:
        states = ck[..., :V * K].unflatten(-1, (V, K)).unflatten(0, (B, -1)).contiguous()
        D.close(states, np.moveaxis(st[:T:64], 0, 1), io, T, "ckpt", size=D.rms(st))
    return y, last, ck


def check_bwd(ops, t, scale=0.3, dlast=True, ckpt=None, seed=90):
    B, T, H, V = t["v"].shape
    io = t["q"].dtype
    dy = U.rand(seed, B, T, H, V, dtype=io)
    dl = U.rand(seed + 1, B, H, V, t["q"].shape[-1], scale=0.3) if dlast else None
    kw = dict(scale=scale, h0=t["h0"], dlast=dl)
    got = ops.delta_scan_bwd(*args(t), dy, **kw)
    if ckpt is not None:
        saved = ops.delta_scan_bwd(*args(t), dy, ckpt=ckpt, **kw)
        for n in got:
            assert torch.equal(got[n], saved[n]), f"{n}: with and without the saved states differ"
    torch.cuda.synchronize()
    h = D.host(t)
    want = M.delta_rule_bwd(scale=scale, dy=U.f64(dy), dlast=U.f64(dl), **h)
    # dg adds up to 64 steps' terms, in quadrature 8 of them
    sizes = dict(dg=8.0 * D.rms(want["dg_terms"]), dbeta=D.rms(want["dbeta_terms"]))
    for n in ("dq", "dk", "dv", "dg", "dbeta", "dh0"):
        D.close(got[n], want[n], io, T, n, size=sizes.get(n))
    return got


# around every edge of the chunk and of the tiles: steps, heads, key and value channels
SIZES = [(1, 1, 1, 1, 8, 8), (2, 2, 1, 2, 16, 24), (1, 15, 2, 2, 64, 64), (2, 16, 1, 3, 72, 16), (1, 17, 1, 1, 128, 128),
         (1, 31, 2, 4, 32, 40), (1, 33, 1, 2, 56, 136), (2, 63, 3, 3, 96, 80), (1, 64, 2, 4, 128, 64), (3, 65, 1, 1, 64, 8),
         (1, 127, 2, 2, 24, 72), (1, 128, 1, 4, 120, 56), (2, 129, 2, 6, 64, 32), (1, 200, 1, 1, 128, 200), (1, 321, 1, 2, 48, 64)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_forward_and_backward(ops, size, dtype):
    B, T, Hk, H, K, V = size
    t = D.delta_inputs(*size, DT[dtype], state=T % 3 != 0, packed=T % 2 == 1, seed=T)
    _, _, ck = check_fwd(ops, t)
    check_bwd(ops, t, dlast=T % 4 != 0, ckpt=ck)


# more chunks and key heads than CUs, one and several blocks of value channels; more workgroups of 64 value channels than
# CUs, where those of 128 are fewer
MANY = [(11, 130, 9, 18, 32, 24), (11, 130, 27, 27, 16, 40), (13, 70, 12, 12, 32, 128), (22, 10, 6, 6, 128, 128)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", MANY, ids=lambda s: "x".join(map(str, s)))
def test_more_work_than_the_gpu_holds(ops, size, dtype):
    t = D.delta_inputs(*size, DT[dtype], seed=5)
    _, _, ck = check_fwd(ops, t)
    check_bwd(ops, t, ckpt=ck)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_sequence(ops, dtype):
    t = D.delta_inputs(1, 3000, 1, 2, 64, 32, DT[dtype], packed=True)
    _, _, ck = check_fwd(ops, t)
    check_bwd(ops, t, ckpt=ck)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_key_again_and_again(ops, dtype):
    """Every step has the same key and full correction: the solve's inverse is a bidiagonal matrix of ones, found from
    a triangle of ones without its large powers."""
    t = D.delta_inputs(1, 190, 1, 2, 64, 64, DT[dtype])
    k = torch.zeros(64, device="cuda")
    k[:4] = 0.5                                        # of length 1, exactly
    t["k"] = k.to(DT[dtype]).expand(1, 190, 1, 64).contiguous()
    t["beta"].fill_(1.0)
    t["g"].zero_()
    check_fwd(ops, t)
    check_bwd(ops, t)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_reflecting_keys(ops, dtype):
    """beta = 2 turns the state over along each unit key; nothing decays."""
    t = D.delta_inputs(1, 130, 1, 2, 64, 32, DT[dtype])
    k = torch.sign(U.rand(9, 1, 130, 1, 64)) * 0.125   # of length 1, exactly
    t["k"] = k.to(DT[dtype])
    t["beta"].fill_(2.0)
    t["g"].zero_()
    t["v"] = t["v"] * 0.1
    check_fwd(ops, t)
    check_bwd(ops, t)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_restarts_and_pads(ops, dtype):
    """g = -inf (or anything below exp's range) restarts the state, beta = g = 0 leaves it alone."""
    t = D.delta_inputs(2, 150, 1, 2, 32, 24, DT[dtype])
    for step, value in ((0, float("-inf")), (37, float("-inf")), (38, -1e30), (64, -200.0), (99, -104.5), (100, -60.0), (149, float("-inf"))):
        t["g"][0, step] = value
    t["g"][1, 70:], t["beta"][1, 70:] = 0.0, 0.0
    y, last, _ = check_fwd(ops, t)
    check_bwd(ops, t)
    alone = ops.delta_scan_fwd(*(t[n][:1, 37:].contiguous() for n in NAMES), scale=0.3)
    assert torch.allclose(alone[0, :60].float(), y[0, 37:97].float(), rtol=2e-2, atol=1e-3 if dtype == "bf16" else 1e-5)
    short, l70 = ops.delta_scan_fwd(*(t[n][1:, :70].contiguous() for n in NAMES), scale=0.3, h0=t["h0"][1:], return_last_state=True)
    assert torch.equal(short[0], y[1, :70])
    D.close(last[1:], U.f64(l70), DT[dtype], 150, "kept state")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_fast_decay(ops, dtype):
    """Decays whose products over a chunk leave fp32's range."""
    t = D.delta_inputs(1, 140, 1, 3, 64, 32, DT[dtype])
    t["g"] = t["g"] * 0 - torch.tensor([0.0, 3.0, 40.0], device="cuda")
    check_fwd(ops, t)
    check_bwd(ops, t)


LENS = [[5], [64], [1, 700, 63, 64, 65, 0, 7], [0, 0, 3], [128, 128], [17, 1, 1, 1, 110, 200, 64, 2], [0]]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", LENS, ids=lambda s: "_".join(map(str, s)))
def test_packed_sequences(ops, lens, dtype):
    """Each sequence by itself; rows before, between and behind them hold NaN, are not read, and stay as they were."""
    before, behind, n = 3, 5, len(lens)
    total = before + sum(lens) + behind
    t = D.delta_inputs(1, total, 2, 4, 64, 40, DT[dtype], packed=True, n=n, seed=len(lens))
    at = np.cumsum([before] + lens)
    starts = torch.tensor(at, dtype=torch.int32, device="cuda")
    dy, dl = U.rand(50, 1, total, 4, 40, dtype=DT[dtype]), U.rand(51, n, 4, 40, 64, scale=0.3)
    for i in list(range(before)) + list(range(total - behind, total)):
        for name in NAMES:
            t[name][0, i] = float("nan")
        dy[0, i] = float("nan")
    y = torch.full((1, total, 4, 40), 7.0, device="cuda").to(DT[dtype])
    ck = torch.full(ops.delta_ckpt_shape(t["q"], t["v"], starts), float("nan"), device="cuda")
    kw = dict(scale=0.3, h0=t["h0"], starts=starts)
    _, last = ops.delta_scan_fwd(*args(t), return_last_state=True, out=y, ckpt_out=ck, **kw)
    got = ops.delta_scan_bwd(*args(t), dy, dlast=dl, **kw)
    saved = ops.delta_scan_bwd(*args(t), dy, dlast=dl, ckpt=ck, **kw)
    torch.cuda.synchronize()
    outside = torch.cat([y[0, :before], y[0, total - behind:]])
    assert bool((outside.float() == 7.0).all())
    for i, m in enumerate(lens):
        one = {name: t[name][:, at[i]:at[i] + m].contiguous() for name in NAMES}
        h0 = t["h0"][i:i + 1]
        ya, la = ops.delta_scan_fwd(*args(one), scale=0.3, h0=h0, return_last_state=True)
        ga = ops.delta_scan_bwd(*args(one), dy[:, at[i]:at[i] + m].contiguous(), dlast=dl[i:i + 1], scale=0.3, h0=h0)
        assert torch.equal(y[:, at[i]:at[i] + m], ya) and torch.equal(last[i:i + 1], la), i
        for name in ("dq", "dk", "dv", "dg", "dbeta"):
            for g in (got, saved):
                assert torch.equal(g[name][:, at[i]:at[i] + m], ga[name]), (i, name)
        for g in (got, saved):
            assert torch.equal(g["dh0"][i:i + 1], ga["dh0"]), i
        if m:
            yo, st = M.delta_rule(scale=0.3, h0=U.f64(h0), **D.host(one))
            D.close(ya, yo, DT[dtype], m, "y", size=0.3 * D.rms(st))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(1, 2, 32, 24), (2, 2, 96, 80)], ids=["32x24", "96x80"])
def test_one_packed_sequence_far_longer_than_the_rest(ops, size, dtype):
    """Long enough for the longest to be cut in time."""
    Hk, H, K, V = size
    lens = [40, 3900, 3, 0, 200, 64, 1, 700]
    total, io = sum(lens), DT[dtype]
    t = D.delta_inputs(1, total, Hk, H, K, V, io, n=len(lens), seed=9)
    at = np.cumsum([0] + lens)
    starts = torch.tensor(at, dtype=torch.int32, device="cuda")
    dy, dl = U.rand(50, 1, total, H, V, dtype=io), U.rand(51, len(lens), H, V, K, scale=0.3)
    ck = torch.empty(ops.delta_ckpt_shape(t["q"], t["v"], starts), device="cuda")
    kw = dict(scale=0.3, h0=t["h0"], starts=starts)
    y, last = ops.delta_scan_fwd(*args(t), return_last_state=True, ckpt_out=ck, **kw)
    got = ops.delta_scan_bwd(*args(t), dy, dlast=dl, **kw)
    saved = ops.delta_scan_bwd(*args(t), dy, dlast=dl, ckpt=ck, **kw)
    torch.cuda.synchronize()
    assert all(torch.equal(got[n], saved[n]) for n in got)
    for i, m in enumerate(lens):
        rows = slice(int(at[i]), int(at[i + 1]))
        one = D.host({name: t[name][:, rows] for name in NAMES})
        h0 = U.f64(t["h0"][i:i + 1])
        yo, st = M.delta_rule(scale=0.3, h0=h0, **one)
        D.close(last[i:i + 1], st[-1], io, m, "last", size=D.rms(st))
        if not m:
            continue
        D.close(y[:, rows], yo, io, m, "y", size=0.3 * D.rms(st) * K ** 0.5 * D.rms(one["q"]))
        want = M.delta_rule_bwd(scale=0.3, dy=U.f64(dy[:, rows]), dlast=U.f64(dl[i:i + 1]), h0=h0, **one)
        sizes = dict(dg=8.0 * D.rms(want["dg_terms"]), dbeta=D.rms(want["dbeta_terms"]))
        for n in ("dq", "dk", "dv", "dg", "dbeta"):
            D.close(got[n][:, rows], want[n], io, m, n, size=sizes.get(n))
        D.close(got["dh0"][i:i + 1], want["dh0"], io, m, "dh0")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(24, 24, 64, 128), (12, 24, 128, 128), (6, 6, 128, 200)], ids=lambda s: "x".join(map(str, s)))
def test_a_cut_sequence_is_its_pieces(ops, size, dtype):
    """A sequence that is cut in time against pieces too short for it, each from the state (gradient) that the one before
    (behind) it leaves.  Each side keeps the tolerance against the exact values, so twice that between them; and each is
    rounded to the outputs' type by itself, v (1 + d) with |d| at most half a step, so they are up to two halves apart:
    |v (1 + d) - v (1 + e)| <= |v| (|d| + |e|)."""
    Hk, H, K, V = size
    T, P, io = 3000, 600, DT[dtype]
    t = D.delta_inputs(1, T, Hk, H, K, V, io, seed=3)
    dy, dl = U.rand(50, 1, T, H, V, dtype=io), U.rand(51, 1, H, V, K, scale=0.3)
    ck = torch.empty(ops.delta_ckpt_shape(t["q"], t["v"]), device="cuda")
    y, last = ops.delta_scan_fwd(*args(t), scale=0.3, h0=t["h0"], return_last_state=True, ckpt_out=ck)
    got = ops.delta_scan_bwd(*args(t), dy, scale=0.3, h0=t["h0"], dlast=dl, ckpt=ck)
    part = lambda i: [t[n][:, i:i + P].contiguous() for n in NAMES]
    states, ys, grads = [t["h0"]], [], []
    for i in range(0, T, P):
        yi, si = ops.delta_scan_fwd(*part(i), scale=0.3, h0=states[-1], return_last_state=True)
        states.append(si)
        ys.append(yi)
    for i in reversed(range(0, T, P)):
        g = ops.delta_scan_bwd(*part(i), dy[:, i:i + P].contiguous(), scale=0.3, h0=states[i // P], dlast=dl)
        dl = g["dh0"]
        grads.insert(0, g)
    want = {n: torch.cat([g[n] for g in grads], 1) for n in ("dq", "dk", "dv", "dg", "dbeta")}
    want.update(y=torch.cat(ys, 1), last=states[-1], dh0=dl)
    got.update(y=y, last=last)
    for n, w in want.items():
        half, w, g = U.HALF_STEP[got[n].dtype], U.f64(w), U.f64(got[n])
        g = g - np.clip(g - w, -half * np.abs(w), half * np.abs(w))            # the second half; close() has the first
        D.close(torch.from_numpy(g).to("cuda"), w, io, T, n, size=2.0 * D.rms(w) * (4.0 if n == "dg" else 1.0), half=half)


def test_many_empty_sequences(ops):
    n = 1000
    at = torch.zeros(n + 1, dtype=torch.int32)
    at[500:] = 70
    t = D.delta_inputs(1, 70, 1, 1, 16, 8, torch.float32, n=n)
    y, last = ops.delta_scan_fwd(*args(t), scale=0.3, h0=t["h0"], starts=at.cuda(), return_last_state=True)
    ya, la = ops.delta_scan_fwd(*args(t), scale=0.3, h0=t["h0"][499:500], return_last_state=True)
    assert torch.equal(y, ya) and torch.equal(last[499:500], la)
    assert torch.equal(last[:499], t["h0"][:499]) and torch.equal(last[500:], t["h0"][500:])


@pytest.mark.parametrize("T", [200, 2000])
def test_starts_out_of_order_stay_inside(ops, T):
    """Bad starts are brought into range on the device: the call ends, and nothing outside the tensors is written."""
    t = D.delta_inputs(1, T, 1, 2, 32, 24, torch.float32, state=False)
    y, guard = U.guarded((1, T, 2, 24), torch.float32)
    for bad in ([0, 150, 40, T], [-50, 10, 4 * T, 3], [2 ** 31 - 1, -2 ** 31, T, 100], [T, T, 0, 0]):
        s = torch.tensor(bad, dtype=torch.int64).to(torch.int32).cuda()
        _, last = ops.delta_scan_fwd(*args(t), starts=s, out=y, return_last_state=True)
        ops.delta_scan_bwd(*args(t), t["v"].contiguous(), starts=s)
        torch.cuda.synchronize()
        guard()
    assert last.shape == (3, 2, 24, 32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_steps(ops, dtype):
    t = D.delta_inputs(2, 0, 1, 2, 16, 8, DT[dtype])
    y, last = ops.delta_scan_fwd(*args(t), h0=t["h0"], return_last_state=True)
    assert y.shape == (2, 0, 2, 8) and torch.equal(last, t["h0"])
    assert not bool(ops.delta_scan_fwd(*args(t), return_last_state=True)[1].any())
    dl = U.rand(3, 2, 2, 8, 16)
    assert torch.equal(ops.delta_scan_bwd(*args(t), y, dlast=dl)["dh0"], dl)
    assert not bool(ops.delta_scan_bwd(*args(t), y)["dh0"].any())


UPDATES = [(1, 1, 1, 8, 8), (3, 1, 2, 16, 24), (2, 2, 6, 32, 40), (5, 1, 1, 40, 64), (2, 2, 4, 64, 136), (1, 3, 3, 96, 80), (2, 2, 4, 128, 128),
           (300, 2, 4, 128, 64), (1, 1, 1, 72, 8)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", UPDATES, ids=lambda s: "x".join(map(str, s)))
def test_one_token(ops, size, dtype):
    B, Hk, H, K, V = size
    t = D.delta_inputs(B, 1, Hk, H, K, V, DT[dtype], seed=B)
    t["g"][0, 0, 0] = float("-inf")
    one = [t[n][:, 0].contiguous() for n in NAMES]
    state, guard = U.guarded((B, H, V, K), torch.float32)
    state.copy_(t["h0"])
    y = ops.delta_state_update(state, *one, scale=0.3)
    torch.cuda.synchronize()
    guard()
    yo, st = M.delta_rule(scale=0.3, **D.host(t))
    D.close(state, st[1], torch.float32, 1, "state")
    D.close(y[:, None], yo, torch.float32, 1, "y", size=0.3 * D.rms(st))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_tokens_continue_a_prompt(ops, dtype):
    t = D.delta_inputs(2, 75, 1, 2, 64, 48, DT[dtype])
    yo, st = M.delta_rule(scale=0.3, **D.host(t))
    size = 0.3 * D.rms(st)
    _, state = ops.delta_scan_fwd(*(t[n][:, :68].contiguous() for n in NAMES), scale=0.3, h0=t["h0"], return_last_state=True)
    for s in range(68, 75):
        ys = ops.delta_state_update(state, *(t[n][:, s].contiguous() for n in NAMES), scale=0.3)
        D.close(ys, yo[:, s], DT[dtype], 75, "token", size=size)
    D.close(state, st[-1], DT[dtype], 75, "state")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_repeats_to_the_bit(ops, dtype):
    t = D.delta_inputs(2, 333, 2, 4, 128, 64, DT[dtype])
    dy = U.rand(7, 2, 333, 4, 64, dtype=DT[dtype])
    first = None
    for _ in range(3):
        y, last = ops.delta_scan_fwd(*args(t), h0=t["h0"], return_last_state=True)
        got = list(ops.delta_scan_bwd(*args(t), dy, h0=t["h0"]).values()) + [y, last]
        first = first or [g.clone() for g in got]
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_gradient_by_differences(ops):
    """Central differences of the kernel's own fp32 forward, in 64-bit sums, along each gradient's signs."""
    t = D.delta_inputs(1, 70, 1, 2, 16, 8, torch.float32)
    dy, dl = U.rand(30, 1, 70, 2, 8), U.rand(31, 1, 2, 8, 16)

    def parts(x):
        y, last = ops.delta_scan_fwd(*args(x), scale=0.3, h0=x["h0"], return_last_state=True)
        return y.double() * dy.double(), last.double() * dl.double()

    got = ops.delta_scan_bwd(*args(t), dy, scale=0.3, h0=t["h0"], dlast=dl)
    # a term of the loss is off by the forward's tolerance relative to the tensor's rms (mixer_util), in quadrature
    noise = 2.0 ** -20 * 2 * (5 * 2) ** 0.5 * float(sum((p * p).sum() for p in parts(t))) ** 0.5
    for n in ("q", "k", "v", "g", "beta", "h0"):
        grad = U.f64(got["d" + n])
        sign = torch.sign(got["d" + n])
        h = 1e-3
        hi, lo = (float(sum(p.sum() for p in parts({**t, n: t[n] + d * sign}))) for d in (h, -h))
        want = float(np.abs(grad).sum())
        # the third derivative: h^2 / 6 of it, its size at most about the third power of the steps' sums along the signs
        assert abs((hi - lo) / (2 * h) - want) <= 2e-2 * want + 4 * 2 ** 0.5 * noise / (2 * h), n


def test_another_stream_and_a_workspace(ops):
    t = D.delta_inputs(1, 200, 1, 2, 64, 64, torch.bfloat16)
    dy = U.rand(8, 1, 200, 2, 64, dtype=torch.bfloat16)
    want, g0 = ops.delta_scan_fwd(*args(t)), ops.delta_scan_bwd(*args(t), dy)
    ws = torch.full((ops.delta_scan_workspace_bytes(t["q"], t["v"]),), 255, dtype=torch.uint8, device="cuda")
    wb = torch.full((ops.delta_scan_bwd_workspace_bytes(t["q"], t["v"]),), 255, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = ops.delta_scan_fwd(*args(t), workspace=ws)
        g1 = ops.delta_scan_bwd(*args(t), dy, workspace=wb)
    side.synchronize()
    assert torch.equal(y, want) and all(torch.equal(g0[n], g1[n]) for n in g0)


def test_captured_in_a_graph(ops):
    t = D.delta_inputs(1, 150, 1, 2, 64, 32, torch.bfloat16)
    dy = U.rand(8, 1, 150, 2, 32, dtype=torch.bfloat16)
    state = t["h0"].clone()
    one = lambda s: [t[n][:, s].contiguous() for n in NAMES]
    tok = one(0)

    def step():
        y, last = ops.delta_scan_fwd(*args(t), h0=t["h0"], return_last_state=True)
        return [y, last, *ops.delta_scan_bwd(*args(t), dy, h0=t["h0"]).values(), ops.delta_state_update(state, *tok)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for r in range(3):
        t["v"].copy_(U.rand(100 + r, 1, 150, 2, 32))
        t["g"].mul_(0.9)
        for a, b in zip(tok, one(r)):
            a.copy_(b)
        before = U.rand(200 + r, 1, 2, 32, 64)
        state.copy_(before)
        graph.replay()
        torch.cuda.synchronize()
        got, after = [o.clone() for o in outs], state.clone()
        state.copy_(before)
        assert all(torch.equal(a, b) for a, b in zip(got, step())) and torch.equal(state, after)


def test_a_nan_stays_in_its_head_and_sequence(ops):
    t = D.delta_inputs(2, 200, 1, 3, 32, 16, torch.float32)
    clean = ops.delta_scan_fwd(*args(t), h0=t["h0"])
    t["v"][1, 130, 2, 5] = float("nan")
    y = ops.delta_scan_fwd(*args(t), h0=t["h0"])
    bad = torch.isnan(y)
    assert not bool(bad[0].any()) and not bool(bad[1, :, :2].any()) and not bool(bad[1, :128].any())
    assert bool(bad[1, 130:, 2, 5].all()) and torch.equal(y[~bad], clean[~bad])


def test_refusals(ops):
    t = D.delta_inputs(1, 20, 1, 2, 16, 8, torch.float32)
    q, k, v, g, beta = args(t)
    bad = [dict(q=q.half()), dict(k=k[..., :8]), dict(v=v.bfloat16()), dict(g=g.bfloat16()), dict(beta=beta[:, :10]), dict(h0=t["h0"][:0]),
           dict(q=q.cpu()), dict(v=v[0]), dict(starts=torch.zeros(2, dtype=torch.int64, device="cuda")),
           dict(starts=torch.zeros(0, dtype=torch.int32, device="cuda")), dict(out=v[:, :10]), dict(ckpt_out=torch.empty(3, device="cuda")),
           dict(starts=torch.zeros(2, dtype=torch.int32))]
    for over in bad:
        kw = {**dict(q=q, k=k, v=v, g=g, beta=beta), **over}
        with pytest.raises(ValueError):
            ops.delta_scan_fwd(**kw)
    late = torch.zeros(321, device="cuda")[1:].view(1, 20, 1, 16)          # contiguous, 4 bytes past a 16-byte address
    with pytest.raises(RuntimeError, match="align"):
        ops.delta_scan_fwd(late, k, v, g, beta)
    with pytest.raises(RuntimeError):
        ops.delta_scan_fwd(q[..., :12].contiguous(), k[..., :12].contiguous(), v, g, beta)
    with pytest.raises(RuntimeError):
        ops.delta_scan_fwd(q, k, v, g, beta, scale=float("nan"))
