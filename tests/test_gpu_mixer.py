"""The gated delta rule and its output norm together, as a block uses them: a
training step with all gradients, packed prompts, then decoding from the state."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_util as U
import mixer_util as D
from oracle import mixer as M

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from selective_scan_ssm_amd import _lib, ops
    _lib.load()
    return ops


B, T, HK, H, K, V = 2, 150, 2, 4, 32, 48
NAMES = ("q", "k", "v", "g", "beta")


def test_training_step(ops):
    """y = group_norm(delta(q, k, v), heads, z): the output and the gradient by every input, in fp32."""
    t = D.delta_inputs(B, T, HK, H, K, V, torch.float32, state=False)
    z, w = U.rand(20, B, T, H * V), 1.0 + 0.1 * U.rand(21, H * V)
    dy = U.rand(22, B, T, H * V)
    args = [t[n] for n in NAMES]
    ck = torch.empty(ops.delta_ckpt_shape(t["q"], t["v"]), device="cuda")
    o = ops.delta_scan_fwd(*args, ckpt_out=ck)
    rows = lambda a: a.reshape(B * T, H * V)
    y, mean, rstd = ops.group_norm(rows(o), H, w, z=rows(z), return_stats=True)
    gn = ops.group_norm_bwd(rows(dy), rows(o), mean, rstd, H, w, z=rows(z))
    gd = ops.delta_scan_bwd(*args, gn["dx"].view(B, T, H, V), ckpt=ck)
    gn_norm = ops.grad_norm([gn["dweight"], gd["dq"]])
    h = {n: U.f64(t[n]) for n in NAMES}
    oo, st = M.delta_rule(scale=K ** -0.5, **h)
    yo, mo, ro = M.group_norm(oo.reshape(B * T, 1, -1), H, U.f64(w), None, U.f64(rows(z))[:, None])
    no = M.group_norm_bwd(U.f64(rows(dy))[:, None], oo.reshape(B * T, 1, -1), mo, ro, U.f64(w), None, U.f64(rows(z))[:, None])
    want = M.delta_rule_bwd(scale=K ** -0.5, dy=no["dx"].reshape(B, T, H, V), **h)
    # the norm divides the mixer's error by the heads' own size: relative to a row's rms it stays, for rows of all sizes
    # up to the largest reciprocal deviation over the smallest
    spread = float(ro.max() * np.sqrt(np.mean(1.0 / ro ** 2)))
    D.close(y, yo[:, 0], torch.float32, T, "y", size=spread * D.rms(yo))
    D.close(gn["dweight"], no["dweight"], torch.float32, T, "dweight", size=spread * D.rms(no["dweight_terms"]))
    D.close(gn["dz"], no["dz"][:, 0], torch.float32, T, "dz", size=spread * D.rms(no["dz"]))
    for n in ("dq", "dk", "dv"):
        D.close(gd[n], want[n], torch.float32, T, n, size=spread * D.rms(want[n]))
    D.close(gd["dg"], want["dg"], torch.float32, T, "dg", size=spread * 8.0 * D.rms(want["dg_terms"]))
    D.close(gd["dbeta"], want["dbeta"], torch.float32, T, "dbeta", size=spread * D.rms(want["dbeta_terms"]))
    total = np.sqrt((no["dweight"] ** 2).sum() + (want["dq"] ** 2).sum())
    assert abs(float(gn_norm) - total) <= 1e-4 * total


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prompts_then_decoding(ops, dtype):
    """Prompts of different lengths packed, then three tokens of each from the states they left, against each
    whole sequence at once."""
    lens, more = [70, 1, 64, 130], 3
    n = len(lens)
    full = [D.delta_inputs(1, m + more, HK, H, K, V, dtype, state=False, seed=10 * i) for i, m in enumerate(lens)]
    prompt = {name: torch.cat([f[name][:, :m] for f, m in zip(full, lens)], 1).contiguous() for name in NAMES}
    starts = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
    y, state = ops.delta_scan_fwd(*(prompt[name] for name in NAMES), starts=starts, return_last_state=True)
    want = [M.delta_rule(scale=K ** -0.5, **{name: U.f64(f[name]) for name in NAMES}) for f in full]
    for i, m in enumerate(lens):
        D.close(y[:, int(starts[i]):int(starts[i + 1])], want[i][0][:, :m], dtype, m, "prompt", size=K ** -0.5 * D.rms(want[i][1]))
    w = torch.ones(H * V, device="cuda")
    for s in range(more):
        tok = [torch.cat([f[name][:, m + s] for f, m in zip(full, lens)]).contiguous() for name in NAMES]
        out = ops.delta_state_update(state, *tok)
        ref = np.concatenate([o[0][:, m + s] for o, m in zip(want, lens)])
        D.close(out, ref, dtype, max(lens), "token", size=K ** -0.5 * max(D.rms(o[1]) for o in want))
        normed = ops.group_norm(out.view(n, H * V), H, w, z=tok[2].view(n, H * V))
        no, _, _ = M.group_norm(U.f64(out).reshape(n, 1, H * V), H, U.f64(w), None, U.f64(tok[2]).reshape(n, 1, H * V))
        assert np.allclose(U.f64(normed), no[:, 0], rtol=U.HALF_STEP[dtype], atol=1e-5)
