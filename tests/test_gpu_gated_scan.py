"""The gated linear recurrence on the GPU against its fp64 definition, within
the rounding bounds derived beside it (oracle/recurrent_block.py)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_util as U
from oracle import recurrent_block as R

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from selective_scan_ssm_amd import _lib, ops
    _lib.load()
    return ops


def inputs(B, T, D, dtype, z=True, state=True, bias=True, packed=False, seed=0):
    n = 3 if z else 2
    if packed:
        proj = U.rand(seed, B, T, n * D, dtype=dtype)
        cols = [proj[..., i * D:(i + 1) * D] for i in range(n)]
    else:
        cols = [U.rand(seed + i, B, T, D, dtype=dtype) for i in range(n)]
    t = dict(x=cols[0], g=cols[1], z=cols[2] if z else None)
    # gates around 0 .. 5: time scales from 2 to some hundred steps
    t["gate_bias"] = (U.rand(seed + 5, D).abs() * 2.5) if bias else None
    t["h0"] = U.rand(seed + 6, B, D) if state else None
    return t


def host(t):
    return {k: U.f64(v) for k, v in t.items()}


def check_fwd(ops, t, **kw):
    B, T, D = t["x"].shape
    y, guard = U.guarded((B, T, D), t["x"].dtype)
    _, last = ops.gated_scan_fwd(t["x"], t["g"], z=t["z"], gate_bias=t["gate_bias"], h0=t["h0"], return_last_state=True,
                                 out=y, **kw)
    torch.cuda.synchronize()
    guard()
    yo, lo, by, bl = R.gated_scan(**host(t), bounds=True)
    U.close(y, yo, by, "y")
    U.close(last, lo, bl, "last")
    return y, last


def check_bwd(ops, t, dlast=True, seed=50):
    B, T, D = t["x"].shape
    dout = U.rand(seed, B, T, D, dtype=t["x"].dtype)
    dl = U.rand(seed + 1, B, D) if dlast else None
    ck = torch.full(ops.gated_ckpt_shape(B, T, D), float("nan"), device="cuda")
    kw = dict(z=t["z"], gate_bias=t["gate_bias"], h0=t["h0"])
    ops.gated_scan_fwd(t["x"], t["g"], ckpt_out=ck, **kw)
    got = ops.gated_scan_bwd(t["x"], t["g"], dout, dlast=dl, ckpt=ck, **kw)
    alone = ops.gated_scan_bwd(t["x"], t["g"], dout, dlast=dl, **kw)
    torch.cuda.synchronize()
    for k, v in got.items():
        assert (v is None) == (alone[k] is None)
        assert v is None or torch.equal(v, alone[k]), f"{k}: with and without the saved states differ"
    want, bound = R.gated_scan_bwd(dout=U.f64(dout), dlast=U.f64(dl), **host(t), bounds=True)
    for k, v in got.items():
        if v is not None:
            U.close(v, want[k], bound[k], k)
    return got


# one step to several blocks, around every tile edge; one channel to several column tiles, odd ones
SIZES = [(1, 1, 1), (2, 1, 64), (1, 2, 3), (3, 15, 65), (2, 16, 128), (1, 17, 130), (2, 63, 64), (1, 64, 256), (2, 65, 5),
         (1, 127, 64), (2, 128, 66), (3, 129, 128), (1, 255, 7), (2, 257, 192), (1, 1000, 321), (2, 1025, 63),
         (1, 2300, 130)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,D", SIZES)
def test_forward(ops, B, T, D, dtype):
    check_fwd(ops, inputs(B, T, D, DT[dtype], z=(T + D) % 2 == 0, state=T % 3 != 0, bias=D % 5 != 0))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,D", SIZES)
def test_backward(ops, B, T, D, dtype):
    check_bwd(ops, inputs(B, T, D, DT[dtype], z=(T + D) % 2 == 1, state=T % 2 == 0, bias=D % 3 != 0), dlast=T % 4 != 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 5, 16, 17, 31, 32, 33, 48, 64, 65])
def test_short_sequences(ops, T, dtype):
    """As many waves as the steps need."""
    for D, z in ((130, True), (65, False)):
        t = inputs(5, T, D, DT[dtype], z=z, seed=T)
        check_fwd(ops, t)
        check_bwd(ops, t)


# enough tiles that bf16 channels are taken in pairs: one tile to a chain, several, more than a state's 64
@pytest.mark.parametrize("B,T,D,z", [(2050, 129, 2, True), (1400, 257, 6, False), (4100, 20, 130, True), (4100, 33, 64, False),
                                     (64, 8200, 2, True), (420, 520, 130, True)])
def test_pairs_of_channels(ops, B, T, D, z):
    t = inputs(B, T, D, torch.bfloat16, z=z, packed=D == 130, seed=T)
    y, last = check_fwd(ops, t)
    # the same channels among others that rule out pairs
    wide = {k: v if v is None or v.dim() < 3 else torch.cat([v, v[..., :1]], -1) for k, v in t.items()}
    wide["gate_bias"], wide["h0"] = (torch.cat([t[k], t[k][..., :1]], -1) for k in ("gate_bias", "h0"))
    x, g = wide.pop("x"), wide.pop("g")
    assert torch.equal(ops.gated_scan_fwd(x, g, **wide)[..., :D], y)
    if B * T * D < 1 << 22:
        check_bwd(ops, t)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,D,z", [(2, 300, 96, True), (1, 150, 33, True), (2, 140, 64, False), (1, 40, 1, True)])
def test_column_ranges_of_one_projection(ops, B, T, D, z, dtype):
    t = inputs(B, T, D, DT[dtype], z=z, packed=True)
    y, last = check_fwd(ops, t)
    got = check_bwd(ops, t)
    c = {k: None if v is None else v.contiguous() for k, v in t.items()}
    y2, last2 = check_fwd(ops, c)
    got2 = check_bwd(ops, c)
    assert torch.equal(y, y2) and torch.equal(last, last2)
    assert all(v is None or torch.equal(v, got2[k]) for k, v in got.items())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_unaligned_bases(ops, dtype):
    """Bases and strides that allow no wide access: every tensor starts one element late."""
    B, T, D = 2, 200, 66
    buf = [U.rand(70 + i, B, T, D + 1, dtype=DT[dtype]) for i in range(3)]
    t = inputs(B, T, D, DT[dtype])
    t["x"], t["g"], t["z"] = (b[..., 1:] for b in buf)
    check_fwd(ops, t)
    check_bwd(ops, t)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_sequence(ops, dtype):
    t = inputs(1, 20000, 64, DT[dtype], z=False)
    check_fwd(ops, t)
    check_bwd(ops, t)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_infinite_gates_pad_and_restart(ops, dtype):
    """g = +inf keeps the state to the end of a padded row; g = -inf starts a
    packed sequence anew; a row that is all padding returns h0."""
    t = inputs(3, 300, 70, DT[dtype], z=False)
    t["g"][0, 137:] = float("inf")
    t["g"][1, 200] = float("-inf")
    t["g"][2] = float("inf")
    y, last = check_fwd(ops, t)
    assert torch.equal(last[2], t["h0"][2])
    short, l137 = ops.gated_scan_fwd(t["x"][:1, :137].contiguous(), t["g"][:1, :137].contiguous(), gate_bias=t["gate_bias"],
                                     h0=t["h0"][:1], return_last_state=True)
    assert torch.equal(y[0, 200], y[0, 299]) and torch.allclose(last[0], l137[0], rtol=1e-6, atol=1e-6)
    alone = ops.gated_scan_fwd(t["x"][1:2, 200:].contiguous(), t["g"][1:2, 200:].contiguous(), gate_bias=t["gate_bias"])
    assert torch.allclose(alone[0].float(), y[1, 200:].float(), rtol=2 * U.HALF_STEP[DT[dtype]], atol=1e-6)
    got = check_bwd(ops, t)
    assert not bool(got["dg"][2].any()) and not bool(got["dx"][2].any())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_extreme_gates(ops, dtype):
    """The type's lowest and largest values, and far gates, beside ordinary ones."""
    t = inputs(1, 260, 64, DT[dtype])
    big = torch.finfo(DT[dtype]).max
    for i, v in enumerate((big, -big, 200.0, -200.0, 88.0, -88.0, 104.0, -104.0, 30.0, -30.0)):
        t["g"][0, i::23, i::7] = v
    t["gate_bias"].zero_()
    check_fwd(ops, t)
    check_bwd(ops, t)


def test_a_nan_stays_in_its_chain_and_after_its_step(ops):
    t = inputs(2, 400, 66, torch.float32, z=False)
    clean = ops.gated_scan_fwd(t["x"], t["g"], gate_bias=t["gate_bias"], h0=t["h0"])
    t["x"][1, 201, 17] = float("nan")
    y = ops.gated_scan_fwd(t["x"], t["g"], gate_bias=t["gate_bias"], h0=t["h0"])
    bad = torch.isnan(y)
    assert bool(bad[1, 201:, 17].all()) and int(bad.sum()) == 400 - 201
    assert torch.equal(torch.where(bad, clean, y), clean)
    t["x"][1, 201, 17], t["g"][0, 5, 2] = 1.0, float("nan")
    assert bool(torch.isnan(ops.gated_scan_fwd(t["x"], t["g"])[0, 5:, 2]).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_empty_sequences(ops, dtype):
    t = inputs(2, 0, 8, DT[dtype])
    y, last = ops.gated_scan_fwd(t["x"], t["g"], z=t["z"], gate_bias=t["gate_bias"], h0=t["h0"], return_last_state=True)
    assert y.shape == (2, 0, 8) and torch.equal(last, t["h0"])
    dl = U.rand(9, 2, 8)
    got = ops.gated_scan_bwd(t["x"], t["g"], y, z=t["z"], gate_bias=t["gate_bias"], dlast=dl)
    assert torch.equal(got["dh0"], dl) and not bool(got["dgate_bias"].any())
    got = ops.gated_scan_bwd(t["x"], t["g"], y, gate_bias=t["gate_bias"])
    assert not bool(got["dh0"].any())
    e = inputs(0, 5, 8, DT[dtype], z=False, state=False)
    assert ops.gated_scan_fwd(e["x"], e["g"]).shape == (0, 5, 8)
    assert not bool(ops.gated_scan_bwd(e["x"], e["g"], e["x"], gate_bias=torch.ones(8, device="cuda"))["dgate_bias"].any())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,D,z", [(1, 1, False), (3, 65, True), (2, 128, False), (256, 520, True)])
def test_one_token(ops, B, D, z, dtype):
    t = inputs(B, 1, D, DT[dtype], z=z)
    state, guard = U.guarded((B, D), torch.float32)
    state.copy_(t["h0"])
    one = {k: t[k][:, 0].contiguous() if t[k] is not None else None for k in ("x", "g", "z")}
    y = ops.gated_state_update(state, one["x"], one["g"], z=one["z"], gate_bias=t["gate_bias"])
    torch.cuda.synchronize()
    guard()
    yo, lo, by, bl = R.gated_scan(**host(t), bounds=True)
    U.close(y, yo[:, 0], by[:, 0], "y")
    U.close(state, lo, bl, "state")


def test_tokens_one_by_one_continue_a_sequence(ops):
    t = inputs(2, 140, 66, torch.float32)
    y, last = ops.gated_scan_fwd(t["x"], t["g"], z=t["z"], gate_bias=t["gate_bias"], h0=t["h0"], return_last_state=True)
    cut = [t[k][:, :130].contiguous() for k in ("x", "g", "z")]
    _, state = ops.gated_scan_fwd(cut[0], cut[1], z=cut[2], gate_bias=t["gate_bias"], h0=t["h0"], return_last_state=True)
    for i in range(130, 140):
        yi = ops.gated_state_update(state, *(t[k][:, i].contiguous() for k in ("x", "g")), z=t["z"][:, i].contiguous(),
                                    gate_bias=t["gate_bias"])
        assert torch.allclose(yi, y[:, i], rtol=1e-5, atol=1e-6)
    assert torch.allclose(state, last, rtol=1e-5, atol=1e-6)


def test_gradient_by_differences(ops):
    """dL/dx along a random direction against central differences of the GPU's
    own forward (fp32, loss summed in fp64)."""
    t = inputs(2, 300, 64, torch.float32)
    dout = U.rand(90, 2, 300, 64)
    got = ops.gated_scan_bwd(t["x"], t["g"], dout, z=t["z"], gate_bias=t["gate_bias"], h0=t["h0"])

    def loss(**kw):
        a = {**t, **kw}
        return (ops.gated_scan_fwd(a["x"], a["g"], z=a["z"], gate_bias=a["gate_bias"], h0=a["h0"]).double() * dout).sum()

    for name in ("x", "g", "z", "gate_bias", "h0"):
        v = U.rand(91, *t[name].shape)
        h = 1e-2
        num = (loss(**{name: t[name] + h * v}) - loss(**{name: t[name] - h * v})) / (2 * h)
        ana = (got["d" + name].double() * v).sum()
        # h^2 truncation (1e-4 of third-derivative terms of order 1) against sums of random sign over 38400 values
        assert abs(num - ana) < 2e-3 * (got["d" + name].double() * v).abs().sum(), name


def test_repeatable_to_the_bit(ops):
    t = inputs(4, 3000, 256, torch.bfloat16)
    dout = U.rand(3, 4, 3000, 256, dtype=torch.bfloat16)
    kw = dict(z=t["z"], gate_bias=t["gate_bias"], h0=t["h0"])
    first = None
    for _ in range(4):
        y, last = ops.gated_scan_fwd(t["x"], t["g"], return_last_state=True, **kw)
        now = [y, last] + list(ops.gated_scan_bwd(t["x"], t["g"], dout, **kw).values())
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(first, now))


def test_graph_replays(ops):
    from test_gpu_graph import replay_matches_eager
    t = inputs(2, 1200, 192, torch.bfloat16)
    t["dout"] = U.rand(8, 2, 1200, 192, dtype=torch.bfloat16)
    t["ck"] = torch.empty(ops.gated_ckpt_shape(2, 1200, 192), device="cuda")

    def fn(t):
        kw = dict(z=t["z"], gate_bias=t["gate_bias"], h0=t["h0"])
        y, last = ops.gated_scan_fwd(t["x"], t["g"], return_last_state=True, ckpt_out=t["ck"], **kw)
        g = ops.gated_scan_bwd(t["x"], t["g"], t["dout"], dlast=last, ckpt=t["ck"], **kw)
        u = ops.gated_scan_bwd(t["x"], t["g"], t["dout"], **kw)
        state = last.clone()
        one = ops.gated_state_update(state, t["x"][:, 0].contiguous(), t["g"][:, 0].contiguous())
        return [y, last, one, state] + list(g.values()) + list(u.values())

    def refill(t, r):
        for k in ("x", "g", "dout"):
            t[k].copy_(torch.randn(t[k].shape, device="cuda"))
    replay_matches_eager(t, fn, refill)


def test_two_streams_at_once_and_a_shared_workspace_in_turn(ops):
    """Calls that overlap on two streams, each with a workspace of its own, and
    calls of different shapes that use one workspace one after the other."""
    a, b = inputs(2, 2600, 128, torch.bfloat16, seed=1), inputs(1, 5000, 64, torch.float32, seed=2)
    run = lambda t, **kw: ops.gated_scan_fwd(t["x"], t["g"], z=t["z"], gate_bias=t["gate_bias"], h0=t["h0"], **kw)
    want = run(a).clone(), run(b).clone()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(3):
        with torch.cuda.stream(s1):
            ya = run(a)
        with torch.cuda.stream(s2):
            yb = run(b)
        got.append((ya, yb))
    torch.cuda.synchronize()
    assert all(torch.equal(x, w) for pair in got for x, w in zip(pair, want))
    ws = torch.full((64 << 20,), 0xff, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        assert torch.equal(run(a, workspace=ws), want[0]) and torch.equal(run(b, workspace=ws), want[1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_wait_that_gives_up_is_reported(ops, dtype):
    """Every hand-over withheld and the waits bounded at 64 polls, from the host:
    all kernels end, the status says so, what depends on another tile is NaN, what
    does not is the usual result, and the next call on the workspace is right."""
    from selective_scan_ssm_amd import _lib
    lib, B, T, D = _lib.load(), 2, 1500, 130
    t = inputs(B, T, D, DT[dtype])
    kw = dict(z=t["z"], gate_bias=t["gate_bias"], h0=t["h0"])
    io = _lib.SSM_BF16 if dtype == "bf16" else _lib.SSM_F32
    need = lib.ssm_gated_scan_bwd_workspace_bytes(B, T, D, io)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    dout = U.rand(3, B, T, D, dtype=DT[dtype])
    ck = torch.empty(ops.gated_ckpt_shape(B, T, D), device="cuda")
    y, last = ops.gated_scan_fwd(t["x"], t["g"], return_last_state=True, ckpt_out=ck, **kw)
    want = ops.gated_scan_bwd(t["x"], t["g"], dout, ckpt=ck, **kw)
    p = lambda v: None if v is None else v.data_ptr()
    stream = torch.cuda.current_stream().cuda_stream
    head = (p(t["x"]), D, p(t["g"]), D, p(t["gate_bias"]), p(t["z"]), D, p(t["h0"]))
    tail = (B, T, D, io, p(ws), need, 64, stream)
    y2, last2 = torch.empty_like(y), torch.empty_like(last)
    assert lib.ssm_testing_gated_fwd_no_handoff(*head, p(y2), p(last2), None, *tail) == 0
    assert ops.scan_status(ws) == _lib.SSM_ERR_WAIT
    assert torch.equal(y2[:, :128], y[:, :128]) and bool(torch.isnan(y2[:, 128:]).all()) and bool(torch.isnan(last2).all())
    g = [torch.empty_like(t["x"]) for _ in range(3)] + [torch.empty(D, device="cuda"), torch.empty(B, D, device="cuda")]
    for saved in (ck, None):
        assert lib.ssm_testing_gated_bwd_no_handoff(*head, p(dout), None, p(saved), *(p(v) for v in g), *tail) == 0
        assert ops.scan_status(ws) == _lib.SSM_ERR_WAIT
        assert bool(torch.isnan(g[0][:, :1408]).all()) and bool(torch.isnan(g[4]).all()) and bool(torch.isnan(g[3]).all())
        assert torch.equal(g[0][:, 1408:], want["dx"][:, 1408:])        # the last tile has nobody to wait for
        assert torch.equal(g[1][:, 1408:], want["dg"][:, 1408:]) == (saved is not None)
    got = ops.gated_scan_bwd(t["x"], t["g"], dout, workspace=ws, **kw)
    assert ops.scan_status(ws) == 0 and all(torch.equal(v, want[k]) for k, v in got.items())
    assert torch.equal(ops.gated_scan_fwd(t["x"], t["g"], workspace=ws, **kw), y) and ops.scan_status(ws) == 0


@pytest.mark.parametrize("T", [1, 128, 129])
@pytest.mark.parametrize("saved", [False, True])
def test_status_of_the_gradient_of_short_sequences(ops, T, saved):
    """The error word has a place of its own in every workspace, also where a
    sequence is one tile and nothing is handed over: the status after a call that
    ran through is OK, whatever the workspace held and whatever the sums are."""
    from selective_scan_ssm_amd import _lib
    B, D = 2, 70
    t = inputs(B, T, D, torch.float32)
    dout = U.rand(3, B, T, D)
    kw = dict(z=t["z"], gate_bias=t["gate_bias"], h0=t["h0"])
    ck = None
    if saved:
        ck = torch.empty(ops.gated_ckpt_shape(B, T, D), device="cuda")
        ops.gated_scan_fwd(t["x"], t["g"], ckpt_out=ck, **kw)
    want = ops.gated_scan_bwd(t["x"], t["g"], dout, ckpt=ck, **kw)
    ws = torch.full((_lib.load().ssm_gated_scan_bwd_workspace_bytes(B, T, D, _lib.SSM_F32),), 255, dtype=torch.uint8, device="cuda")
    got = ops.gated_scan_bwd(t["x"], t["g"], dout, ckpt=ck, workspace=ws, **kw)
    assert ops.scan_status(ws) == 0
    assert all(torch.equal(v, want[k]) for k, v in got.items())


def test_offsets_past_32_bits(ops):
    """A batch whose projection spans 9 GB: every batch row equals a call on that row alone."""
    B, T, D = 3, 50000, 5120
    proj = torch.empty(B, T, 3 * D, dtype=torch.bfloat16, device="cuda")
    torch.manual_seed(5)
    for i in range(B):
        proj[i].normal_()
    x, g, z = (proj[..., i * D:(i + 1) * D] for i in range(3))
    assert proj.numel() * 2 > 1 << 32
    y, last = ops.gated_scan_fwd(x, g, z=z, return_last_state=True)
    for i in (0, B - 1):
        yi, li = ops.gated_scan_fwd(x[i:i + 1].contiguous(), g[i:i + 1].contiguous(), z=z[i:i + 1].contiguous(),
                                    return_last_state=True)
        assert torch.equal(yi[0], y[i]) and torch.equal(li[0], last[i])
        del yi, li
    got = ops.gated_scan_bwd(x, g, y, z=z)
    i = B - 1
    gi = ops.gated_scan_bwd(x[i:].contiguous(), g[i:].contiguous(), y[i:], z=z[i:].contiguous())
    assert all(torch.equal(got[k][i], gi[k][0]) for k in ("dx", "dg", "dz", "dh0"))


def test_refusals(ops):
    t = inputs(2, 8, 64, torch.bfloat16)
    x, g = t["x"], t["g"]
    for bad in (lambda: ops.gated_scan_fwd(x.half(), g.half()), lambda: ops.gated_scan_fwd(x, g.float()),
                lambda: ops.gated_scan_fwd(x, g[:, :4]), lambda: ops.gated_scan_fwd(x.cpu(), g),
                lambda: ops.gated_scan_fwd(x.transpose(1, 2), g.transpose(1, 2)),
                lambda: ops.gated_scan_fwd(x[:, :, :1].expand(2, 8, 64), g), lambda: ops.gated_scan_fwd(x[:, ::2], g[:, ::2][:1]),
                lambda: ops.gated_scan_fwd(x[:, :1].expand(2, 8, 64), g), lambda: ops.gated_scan_fwd(x, g, h0=t["h0"][:1]),
                lambda: ops.gated_scan_fwd(x, g, gate_bias=t["gate_bias"].bfloat16()),
                lambda: ops.gated_scan_fwd(x, g, ckpt_out=torch.empty(2, 1, 63, device="cuda")),
                lambda: ops.gated_scan_bwd(x, g, x[:, :, :32]), lambda: ops.gated_state_update(t["h0"], x, g),
                lambda: ops.gated_state_update(t["h0"].bfloat16(), x[:, 0].contiguous(), g[:, 0].contiguous())):
        with pytest.raises((ValueError, RuntimeError)):
            bad()
    with pytest.raises(RuntimeError, match="ALIAS"):
        ops.gated_scan_fwd(x, g, out=x)


@pytest.mark.parametrize("B,T,D", [(40000, 16, 4096), (65535, 130, 128)])
def test_many_short_sequences(ops, B, T, D):
    """Millions of one-wave tiles over 2.6e9 elements, and the largest batch: the first and last sequences, and the sums
    over all of them."""
    make = lambda: torch.empty(B, T, D, dtype=torch.bfloat16, device="cuda").normal_()
    x, g, dout = make(), make(), make()
    bias = U.rand(1, D).abs() * 2
    y, last = ops.gated_scan_fwd(x, g, gate_bias=bias, return_last_state=True)
    got = ops.gated_scan_bwd(x, g, dout, gate_bias=bias)
    for s in (slice(0, 3), slice(B - 3, B)):
        t = dict(x=x[s], g=g[s], z=None, gate_bias=bias, h0=None)
        yo, lo, by, bl = R.gated_scan(**host(t), bounds=True)
        U.close(y[s], yo, by, "y")
        U.close(last[s], lo, bl, "last")
        want, bound = R.gated_scan_bwd(dout=U.f64(dout[s]), **host(t), bounds=True)
        for k in ("dx", "dg", "dh0"):
            U.close(got[k][s], want[k], bound[k], k)
    total = got["dg"].sum((0, 1), dtype=torch.float64)
    # dg rounds to bf16 after it is summed: half a step of each, in quadrature over B x T values of either sign, times 8;
    # and the fp32 additions, under 2^12 on any path
    size = got["dg"].double().square().sum((0, 1)).sqrt() if got["dg"].numel() < 1 << 31 else \
        torch.stack([c.double().square().sum((0, 1)) for c in got["dg"].split(4096)]).sum(0).sqrt()
    tol = 8 * 2.0 ** -8 * size + 2.0 ** -12 * got["dg"].abs().sum((0, 1), dtype=torch.float64)
    assert bool(((got["dgate_bias"].double() - total).abs() <= tol).all())


def test_bias_gradient_of_the_largest_batch(ops):
    """A thousand tiles' sums one after the other in each stripe, of one large value and small ones that are lost."""
    B = 65535
    dg = torch.where(torch.arange(B) < 64, 1.0, 0.99 * 2.0 ** -24).view(B, 1, 1).expand(B, 1, 3)
    x, g, bias = -torch.ones(B, 1, 3, device="cuda"), torch.zeros(B, 1, 3, device="cuda"), torch.zeros(3, device="cuda")
    dout = (4.0 * dg).cuda().contiguous()
    got = ops.gated_scan_bwd(x, g, dout, gate_bias=bias)
    want, bound = R.gated_scan_bwd(U.f64(x), U.f64(g), U.f64(dout), gate_bias=U.f64(bias), bounds=True)
    for k in ("dx", "dg", "dgate_bias", "dh0"):
        U.close(got[k], want[k], bound[k], k)


def test_a_small_workspace_is_refused(ops):
    """Not replaced: its status word would never be written."""
    t = inputs(2, 300, 64, torch.bfloat16)
    kw = dict(z=t["z"], gate_bias=t["gate_bias"], h0=t["h0"])
    dout = U.rand(1, 2, 300, 64, dtype=torch.bfloat16)
    for fn, need in ((lambda ws: ops.gated_scan_fwd(t["x"], t["g"], workspace=ws, **kw), ops.gated_scan_workspace_bytes),
                     (lambda ws: ops.gated_scan_bwd(t["x"], t["g"], dout, workspace=ws, **kw)["dx"], ops.gated_scan_bwd_workspace_bytes)):
        n = need(2, 300, 64, torch.bfloat16)
        ws = torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")
        with pytest.raises(ValueError, match="are needed"):
            fn(ws[:n - 1])
        assert bool((ws == 0xff).all())
        assert torch.equal(fn(ws), fn(None)) and ops.scan_status(ws) == 0


def test_gradient_by_differences_along_its_signs(ops):
    """As above where no terms cancel: a gradient that is off by 1% fails (test_block_oracle.py shows that it would)."""
    t = {k: v for k, v in inputs(2, 300, 64, torch.float32).items()}
    dout, dlast = U.rand(90, 2, 300, 64), U.rand(91, 2, 64)
    got = ops.gated_scan_bwd(t["x"], t["g"], dout, z=t["z"], gate_bias=t["gate_bias"], h0=t["h0"], dlast=dlast)

    def loss(a):
        y, last = ops.gated_scan_fwd(a["x"], a["g"], z=a["z"], gate_bias=a["gate_bias"], h0=a["h0"], return_last_state=True)
        return float((y.double() * dout).sum() + (last.double() * dlast).sum())

    _, _, ey, el = R.gated_scan(**host(t), bounds=True)
    noise = np.sqrt(((ey * U.f64(dout)) ** 2).sum() + ((el * U.f64(dlast)) ** 2).sum())
    for name in ("x", "g", "z", "gate_bias", "h0"):
        off, allowed = U.along_its_signs(loss, t, name, got["d" + name].double(), 0.02, noise)
        assert float(off) <= float(allowed) < 0.006 * float(got["d" + name].double().abs().sum()), name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 3])
def test_a_few_steps_far_apart(ops, dtype, T):
    """A few steps of each sequence far apart in one wide buffer: 100 MB and more from row to row."""
    B, D = 3, 66
    flat = torch.empty(B * 150 << 20, dtype=DT[dtype], device="cuda")
    step = flat.numel() // (B * T)
    x, g, z = (flat.as_strided((B, T, D), (T * step, step, 1), i * 1000 + 7) for i in range(3))
    for i, t in enumerate((x, g, z)):
        t.copy_(U.rand(i, B, T, D))
    assert 128 * step * x.element_size() >= 1 << 31               # more than 128 such rows could span
    t = dict(x=x, g=g, z=z, gate_bias=U.rand(5, D).abs(), h0=U.rand(6, B, D))
    check_fwd(ops, t)
    check_bwd(ops, t)
