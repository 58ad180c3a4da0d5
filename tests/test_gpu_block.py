"""The gated recurrent block's operators together, as a training step and a
decode loop use them: norm -> projections -> recurrence -> gradients -> clip,
against fp64 autograd on the CPU."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_util as U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from selective_scan_ssm_amd import _lib, ops
    _lib.load()
    return ops


def reference(x, res, w, W, bias, h0, dout):
    """Two values of the step in fp64 on the CPU: outputs and gradients by autograd."""
    x, res, w, W, bias, h0 = (t.detach().double().cpu().requires_grad_() for t in (x, res, w, W, bias, h0))
    r = x + res
    n = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + 1e-5) * w
    p = n @ W.t()
    xs, g, z = p.chunk(3, -1)
    a = torch.sigmoid(g + bias)
    h, ys = h0, []
    for t in range(x.shape[1]):
        h = a[:, t] * h + (1 - a[:, t]) * xs[:, t]
        ys.append(h * torch.nn.functional.silu(z[:, t]))
    y = torch.stack(ys, 1)
    (y * dout.double().cpu()).sum().backward()
    return y, h, [t.grad for t in (x, w, W, bias, h0)]


def test_a_training_step(ops):
    B, T, dm, di = 2, 200, 96, 64
    x, res, w = U.rand(1, B, T, dm), U.rand(2, B, T, dm), 1.0 + 0.1 * U.rand(3, dm)
    W, bias, h0 = U.rand(4, 3 * di, dm, scale=0.1), U.rand(5, di).abs() * 2, U.rand(6, B, di)
    dout = U.rand(7, B, T, di)
    n, r = ops.add_rms_norm(x, w, res)
    proj = n @ W.t()
    xs, g, z = proj.chunk(3, -1)
    ck = torch.empty(ops.gated_ckpt_shape(B, T, di), device="cuda")
    y, last = ops.gated_scan_fwd(xs, g, z=z, gate_bias=bias, h0=h0, return_last_state=True, ckpt_out=ck)
    got = ops.gated_scan_bwd(xs, g, dout, z=z, gate_bias=bias, h0=h0, ckpt=ck)
    dproj = torch.cat([got["dx"], got["dg"], got["dz"]], -1)
    dW = dproj.reshape(-1, 3 * di).t() @ n.reshape(-1, dm)
    back = ops.add_rms_norm_bwd((dproj @ W).contiguous(), r, w)
    yo, lo, (dx, dw, dWo, db, dh0) = reference(x, res, w, W, bias, h0, dout)
    # fp32 throughout: products over 96 and 64 terms and 400-row sums around it, each worth some 10^-6 of the largest
    for name, a, b in (("y", y, yo), ("last", last, lo), ("dx", back["dx"], dx), ("dw", back["dweight"], dw), ("dW", dW, dWo),
                       ("dbias", got["dgate_bias"], db), ("dh0", got["dh0"], dh0)):
        b = b.detach().numpy()
        assert np.abs(U.f64(a) - b).max() <= 2e-5 * np.abs(b).max(), name
    params = [back["dweight"], dW, got["dgate_bias"]]
    want = float(torch.sqrt(sum((t.double() ** 2).sum() for t in (dw, dWo, db))))
    norm = ops.clip_grads(params, want / 3)
    assert abs(float(norm) - want) <= 2e-5 * want
    assert abs(float(ops.grad_norm(params)) - want / 3) <= 2e-5 * want


def test_decode_continues_a_prefill(ops):
    """Prefill 150 tokens, then ten one by one, with the norm in bf16 and its
    8-bit form in front: the states and outputs of one long prefill."""
    B, T, dm, di = 3, 160, 128, 64
    bf = torch.bfloat16
    x, w = U.rand(1, B, T, dm, dtype=bf), 1.0 + 0.1 * U.rand(3, dm)
    W, bias = U.rand(4, 3 * di, dm, scale=0.1).to(bf), U.rand(5, di).abs() * 2
    def proj(xt):
        q, s, _ = ops.add_rms_norm_quant(xt, w)
        y, _ = ops.add_rms_norm(xt, w)
        # the 8-bit rows stand for y to within half a step of e4m3
        assert bool(((q.float() * s[..., None] - y.float()).abs() <= y.float().abs() * (2 ** -4 + 2 ** -7) + s[..., None] * 2 ** -9).all())
        return ((q.float() * s[..., None]) @ W.float().t()).to(bf).chunk(3, -1)
    xs, g, z = proj(x)
    y, last = ops.gated_scan_fwd(xs, g, z=z, gate_bias=bias, return_last_state=True)
    xs1, g1, z1 = proj(x[:, :150].contiguous())
    _, state = ops.gated_scan_fwd(xs1, g1, z=z1, gate_bias=bias, return_last_state=True)
    for t in range(150, 160):
        xt, gt, zt = (v.contiguous() for v in proj(x[:, t]))
        yt = ops.gated_state_update(state, xt, gt, z=zt, gate_bias=bias)
        # the projection's fp32 sums may round to bf16 differently by one step for another batch size
        assert torch.allclose(yt.float(), y[:, t].float(), rtol=2 ** -5, atol=2e-2)
    assert torch.allclose(state, last, rtol=2 ** -6, atol=1e-2)
