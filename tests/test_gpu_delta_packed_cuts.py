"""Packed sequences several of which are cut in time: their segments, borders and joins, with rows outside of all, and a
captured call whose starts change between replays."""
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


MIXES = [(70, [0, 1500, 0, 0, 2100, 64, 900, 1, 1300], 130), (0, [3000, 1, 63, 65, 1], 0), (5, [900, 900, 900, 900], 1), (1, [64, 64, 64, 2600, 64], 0)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(1, 2, 32, 24), (2, 2, 72, 136)], ids=["32x24", "72x136"])
@pytest.mark.parametrize("mix", range(len(MIXES)))
def test_several_cut_sequences(ops, mix, size, dtype):
    """Every sequence against the definition; the rows outside of all hold NaN, and stay as they were in the output."""
    before, lens, behind = MIXES[mix]
    Hk, H, K, V = size
    total, io, n = before + sum(lens) + behind, DT[dtype], len(lens)
    t = D.delta_inputs(1, total, Hk, H, K, V, io, packed=True, n=n, seed=mix)
    at = np.cumsum([before] + lens)
    starts = torch.tensor(at, dtype=torch.int32, device="cuda")
    dy, dl = U.rand(50, 1, total, H, V, dtype=io), U.rand(51, n, H, V, K, scale=0.3)
    for rows in (slice(0, before), slice(total - behind, total)):
        for name in NAMES:
            t[name][:, rows] = float("nan")
        dy[:, rows] = float("nan")
    y = torch.full((1, total, H, V), 7.0, device="cuda").to(io)
    ck = torch.full(ops.delta_ckpt_shape(t["q"], t["v"], starts), float("nan"), device="cuda")
    args, kw = [t[x] for x in NAMES], dict(scale=0.3, h0=t["h0"], starts=starts)
    _, last = ops.delta_scan_fwd(*args, return_last_state=True, out=y, ckpt_out=ck, **kw)
    got = ops.delta_scan_bwd(*args, dy, dlast=dl, **kw)
    saved = ops.delta_scan_bwd(*args, dy, dlast=dl, ckpt=ck, **kw)
    torch.cuda.synchronize()
    inside = slice(before, total - behind)
    assert all(torch.equal(got[x][:, inside], saved[x][:, inside]) for x in ("dq", "dk", "dv", "dg", "dbeta"))
    assert torch.equal(got["dh0"], saved["dh0"])
    assert bool((torch.cat([y[0, :before], y[0, total - behind:]]).float() == 7.0).all())
    for i, m in enumerate(lens):
        rows = slice(int(at[i]), int(at[i + 1]))
        one = D.host({x: t[x][:, rows] for x in NAMES})
        h0 = U.f64(t["h0"][i:i + 1])
        yo, st = M.delta_rule(scale=0.3, h0=h0, **one)
        D.close(last[i:i + 1], st[-1], io, m, f"last {i}", size=D.rms(st))
        if not m:
            assert torch.equal(got["dh0"][i], dl[i])
            continue
        D.close(y[:, rows], yo, io, m, f"y {i}", size=0.3 * D.rms(st) * K ** 0.5 * D.rms(one["q"]))
        want = M.delta_rule_bwd(scale=0.3, dy=U.f64(dy[:, rows]), dlast=U.f64(dl[i:i + 1]), h0=h0, **one)
        sizes = dict(dg=8.0 * D.rms(want["dg_terms"]), dbeta=D.rms(want["dbeta_terms"]))
        for x in ("dq", "dk", "dv", "dg", "dbeta"):
            D.close(got[x][:, rows], want[x], io, m, f"{x} {i}", size=sizes.get(x))
        D.close(got["dh0"][i:i + 1], want["dh0"], io, m, f"dh0 {i}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_captured_with_other_starts(ops, dtype):
    """The lengths are read on the device: a replay with others gives what an eager call on them does, to the bit."""
    io, total, n = DT[dtype], 4000, 6
    t = D.delta_inputs(1, total, 1, 2, 64, 40, io, n=n)
    dy = U.rand(8, 1, total, 2, 40, dtype=io)
    cuts = [[0, 10, 3000, 3000, 3064, 3900, 4000], [0, 0, 0, 0, 0, 0, 4000], [0, 700, 1400, 2100, 2800, 3500, 4000], [100, 101, 1500, 1564, 3600, 3601, 3700]]
    starts = torch.tensor(cuts[2], dtype=torch.int32, device="cuda")
    args, kw = [t[x] for x in NAMES], dict(scale=0.3, h0=t["h0"], starts=starts)
    y = torch.zeros(1, total, 2, 40, dtype=io, device="cuda")

    def step():
        _, last = ops.delta_scan_fwd(*args, return_last_state=True, out=y, **kw)
        return [last, *ops.delta_scan_bwd(*args, dy, **kw).values()]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for c in cuts + cuts[:1]:
        starts.copy_(torch.tensor(c, dtype=torch.int32))
        rows = slice(c[0], c[-1])
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got, first = [o.clone() for o in outs], y.clone()
        y.zero_()
        want = step()
        assert torch.equal(first, y)
        for a, b in zip(got, want):
            a, b = (a[:, rows], b[:, rows]) if a.shape[:2] == (1, total) else (a, b)
            assert torch.equal(a, b)
