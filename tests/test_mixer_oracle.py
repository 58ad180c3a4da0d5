"""The fp64 definitions of the gated delta rule and of the group norm
(oracle/mixer.py) against facts of their own: hand-worked chains, the
reflections that the rule is made of, continuation, differences, autograd."""
import numpy as np
import pytest
import torch

from oracle import mixer as M


def rand(rng, *shape):
    return rng.standard_normal(shape)


def delta_inputs(rng, B=2, T=7, Hk=1, H=2, K=3, V=4):
    k = rand(rng, B, T, Hk, K)
    return dict(q=rand(rng, B, T, Hk, K), k=k / np.linalg.norm(k, axis=-1, keepdims=True), v=rand(rng, B, T, H, V),
                g=-np.abs(rand(rng, B, T, H)), beta=M.sigmoid(rand(rng, B, T, H)), h0=rand(rng, B, H, V, K))


def test_hand_worked_chain():
    # one channel each: s = 2 e^0 = 2, r = 3 - 2 = 1, s = 2 + 0.5 = 2.5; then s = 1.25, r = 4 - 2 * 1.25 = 1.5, s = 1.25 + 3 * 2 * 0.25
    one = lambda *a: np.array(a).reshape(1, 2, 1, 1)
    y, st = M.delta_rule(one(1.0, 3.0), one(1.0, 2.0), one(3.0, 4.0), np.array([0.0, np.log(0.5)]).reshape(1, 2, 1),
                         np.array([0.5, 0.25]).reshape(1, 2, 1), 2.0, h0=np.full((1, 1, 1, 1), 2.0))
    assert np.allclose(st[:, 0, 0, 0, 0], [2.0, 2.5, 2.0], rtol=1e-15)
    assert np.allclose(y[0, :, 0, 0], [2 * 2.5, 2 * 3 * 2.0], rtol=1e-15)


def test_full_correction_stores_the_value_under_its_key():
    rng = np.random.default_rng(1)
    i = delta_inputs(rng)
    i["beta"][:] = 1.0
    i["q"] = i["k"]
    y, _ = M.delta_rule(scale=1.0, **i)
    assert np.allclose(y, i["v"], atol=1e-13)          # what a unit key was given is what it returns


def test_steps_are_products():
    rng = np.random.default_rng(2)
    i = delta_inputs(rng, B=1, H=1, V=2)
    _, st = M.delta_rule(scale=1.0, **i)
    want = i["h0"][0, 0]
    for t in range(7):
        k = i["k"][0, t, 0]
        want = np.exp(i["g"][0, t, 0]) * want @ (np.eye(3) - i["beta"][0, t, 0] * np.outer(k, k)) \
            + i["beta"][0, t, 0] * np.outer(i["v"][0, t, 0], k)
    assert np.allclose(st[7, 0, 0], want, rtol=1e-13)


def test_continuation_and_shared_heads():
    rng = np.random.default_rng(3)
    i = delta_inputs(rng, T=9, Hk=2, H=4)
    y, st = M.delta_rule(scale=0.7, **i)
    cut = lambda a, b: {n: t[:, a:b] for n, t in i.items() if n != "h0"}
    y1, s1 = M.delta_rule(scale=0.7, h0=i["h0"], **cut(0, 4))
    y2, s2 = M.delta_rule(scale=0.7, h0=s1[-1], **cut(4, 9))
    assert np.array_equal(np.concatenate([y1, y2], 1), y) and np.array_equal(s2[-1], st[-1])
    one = {n: (t[:, :, 1:2] if n in "qk" else t[:, 2:3] if n == "h0" else t[:, :, 2:3]) for n, t in i.items()}
    assert np.array_equal(M.delta_rule(scale=0.7, **one)[0][:, :, 0], y[:, :, 2])


@pytest.mark.parametrize("state", [False, True])
def test_delta_gradient_by_differences(state):
    rng = np.random.default_rng(4)
    i = delta_inputs(rng, T=4, Hk=1, H=2, K=2, V=3)
    if not state:
        i.pop("h0")
    dy, dlast = rand(rng, 2, 4, 2, 3), rand(rng, 2, 2, 3, 2)

    def loss(**kw):
        y, st = M.delta_rule(scale=0.6, **kw)
        return (y * dy).sum() + (st[-1] * dlast).sum()

    got = M.delta_rule_bwd(scale=0.6, dy=dy, dlast=dlast, **i)
    for name, value in i.items():
        for at in np.ndindex(value.shape):
            lo, hi = value.copy(), value.copy()
            lo[at] -= 1e-5
            hi[at] += 1e-5
            want = (loss(**{**i, name: hi}) - loss(**{**i, name: lo})) / 2e-5
            assert abs(got["d" + name][at] - want) < 1e-8, (name, at)


def test_group_norm_by_hand():
    y, mean, rstd = M.group_norm(np.array([[[1.0, 3.0, 5.0, 5.0]]]), 2, eps=0.0 + 1e-300)
    assert np.allclose(mean, [[2.0, 5.0]]) and np.isclose(rstd[0, 0], 1.0)
    assert np.allclose(y[0, 0, :2], [-1.0, 1.0]) and np.all(y[0, 0, 2:] == 0.0)


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("gate", [False, True])
def test_group_norm_against_autograd(silu, gate):
    rng = np.random.default_rng(5)
    N, R, C, G = 3, 5, 12, 4
    x, w, b, dy = rand(rng, N, R, C), rand(rng, C), rand(rng, C), rand(rng, N, R, C)
    z = rand(rng, N, R, C) if gate else None
    t = {n: torch.from_numpy(a).requires_grad_() for n, a in dict(x=x, w=w, b=b, z=z).items() if a is not None}
    a = torch.nn.functional.group_norm(t["x"].movedim(-1, 1), G, t["w"], t["b"], eps=1e-5).movedim(1, -1)
    y = torch.nn.functional.silu(a) if silu else a
    if gate:
        y = y * torch.nn.functional.silu(t["z"])
    (y * torch.from_numpy(dy)).sum().backward()
    yo, mean, rstd = M.group_norm(x, G, w, b, z, silu)
    assert np.allclose(yo, y.detach().numpy(), rtol=1e-11, atol=1e-12)
    o = M.group_norm_bwd(dy, x, mean, rstd, w, b, z, silu)
    for name, n in (("dx", "x"), ("dweight", "w"), ("dbias", "b")) + ((("dz", "z"),) if gate else ()):
        assert np.allclose(o[name], t[n].grad.numpy(), rtol=1e-10, atol=1e-11), name
