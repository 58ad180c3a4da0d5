"""The torch wrappers of the gated delta rule and of the group norm where no GPU
is needed: the package's exports, shapes, workspace sizes, refusals."""
import os

import pytest

torch = pytest.importorskip("torch")

from selective_scan_ssm_amd import _lib


@pytest.fixture(scope="module")
def ops():
    if not os.path.exists(_lib.LIB_PATH):
        from selective_scan_ssm_amd import build
        build.build()
    from selective_scan_ssm_amd import ops
    return ops


def test_exports(ops):
    import selective_scan_ssm_amd as package
    for name in ("delta_scan_fwd", "delta_scan_bwd", "delta_state_update", "delta_ckpt_shape", "delta_scan_workspace_bytes",
                 "delta_scan_bwd_workspace_bytes", "group_norm", "group_norm_bwd"):
        assert name in package.__all__ and getattr(package, name) is getattr(ops, name), name


def test_shapes_and_sizes(ops):
    lib = _lib.load()
    q, v = torch.empty(2, 130, 2, 8), torch.empty(2, 130, 4, 16)
    assert ops.delta_ckpt_shape(q, v) == (6, 4, 16 * (8 + 64))
    starts = torch.zeros(6, dtype=torch.int32)
    assert ops.delta_ckpt_shape(q[:1], v[:1], starts) == (2 + 5, 4, 16 * (8 + 64))
    assert ops.delta_ckpt_shape(q[:1, :0], v[:1, :0], starts) == (0, 4, 16 * (8 + 64))
    assert ops.delta_scan_workspace_bytes(q, v) == lib.ssm_delta_scan_workspace_bytes(2, 130, 0, 2, 2, 4, 8, 16, 0)
    assert ops.delta_scan_bwd_workspace_bytes(q, v, saved=True) == lib.ssm_delta_scan_bwd_workspace_bytes(2, 130, 0, 2, 2, 4, 8, 16, 1, 0)
    with pytest.raises(RuntimeError, match="invalid arguments"):
        ops.delta_scan_workspace_bytes(q, v, starts)                     # packed sequences are one batch row
    with pytest.raises(ValueError, match="one value more"):
        ops.delta_ckpt_shape(q[:1], v[:1], starts[:0])


def test_cpu_tensors_are_refused(ops):
    t = torch.zeros(1, 4, 2, 8)
    with pytest.raises(ValueError, match="GPU tensor"):
        ops.delta_scan_fwd(t, t, t, t[..., 0], t[..., 0])
    with pytest.raises(ValueError, match="GPU tensor"):
        ops.delta_state_update(torch.zeros(1, 2, 8, 8), t[:, 0], t[:, 0], t[:, 0], t[:, 0, :, 0], t[:, 0, :, 0])
    with pytest.raises(ValueError, match="GPU tensor"):
        ops.group_norm(t[0, 0], 2)


def test_heads_views(ops):
    """Which strided views of (batch, seqlen, heads, width) a call takes."""
    dev, f = torch.device("cpu"), torch.float32
    at = lambda t: ops._heads(t, "q", f, t.shape, dev)
    # strides are looked at on stand-ins that claim to be on a GPU
    assert at(torch.zeros(2, 5, 3, 4))[1] == 12

    class View:
        is_cuda, dtype, device = True, f, dev

        def __init__(self, t):
            self.t, self.shape = t, t.shape

        def __getattr__(self, name):
            return getattr(self.t, name)

    wide = torch.zeros(2, 5, 40)
    assert ops._heads(View(wide[..., 8:20].unflatten(-1, (3, 4))), "q", f, torch.Size((2, 5, 3, 4)), dev)[1] == 40
    assert ops._heads(View(wide[:, :1, 8:20].unflatten(-1, (3, 4))), "q", f, torch.Size((2, 1, 3, 4)), dev)[1] == 200
    for bad in (torch.zeros(2, 5, 4, 3).transpose(2, 3), torch.zeros(2, 3, 5, 4).transpose(1, 2), wide[:, :4, :12].unflatten(-1, (3, 4)),
                torch.zeros(2, 5, 3, 8)[..., :4]):
        with pytest.raises(ValueError):
            ops._heads(View(bad), "q", f, bad.shape, dev)
