"""The torch wrappers of the gated recurrent block where no GPU is needed: the
package's exports, workspaces and their sizes."""
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


def test_a_workspace_that_is_read_for_its_status_is_not_replaced(ops):
    dev = torch.device("cpu")
    small, large = torch.empty(100, dtype=torch.uint8), torch.empty(300, dtype=torch.uint8)
    with pytest.raises(ValueError, match="100 bytes, 200 are needed"):
        ops._scratch(200, "f", small, dev, status=True)
    assert ops._scratch(200, "f", large, dev, status=True)[0] is large
    assert ops._scratch(200, "f", None, dev, status=True)[0].numel() == 200
    assert ops._scratch(200, "f", small, dev)[0].numel() == 200          # no status: replaced, as in the other wrappers
    assert ops._scratch(0, "f", small, dev, status=True) == (None, None)


def test_workspace_sizes(ops):
    lib = _lib.load()
    for dtype, io in ((torch.float32, 0), (torch.bfloat16, 1)):
        for shape in ((1, 128, 64), (2, 300, 65), (0, 300, 8)):
            assert ops.gated_scan_workspace_bytes(*shape, dtype) == lib.ssm_gated_scan_workspace_bytes(*shape, io)
            assert ops.gated_scan_bwd_workspace_bytes(*shape, dtype) == lib.ssm_gated_scan_bwd_workspace_bytes(*shape, io)
    assert ops.gated_scan_workspace_bytes(1, 128, 64, torch.float32) == 0
    for fn in (ops.gated_scan_workspace_bytes, ops.gated_scan_bwd_workspace_bytes):
        with pytest.raises(RuntimeError, match="invalid arguments"):
            fn(-1, 128, 64, torch.float32)


def test_the_package_exports_what_the_block_needs(ops):
    import selective_scan_ssm_amd as package
    for name in ("gated_scan_fwd", "gated_scan_bwd", "gated_state_update", "gated_ckpt_shape", "gated_scan_workspace_bytes",
                 "gated_scan_bwd_workspace_bytes", "add_rms_norm", "add_rms_norm_quant", "add_rms_norm_bwd", "grad_norm",
                 "clip_grads", "scan_status"):
        assert name in package.__all__ and getattr(package, name) is getattr(ops, name), name
    assert package.gated_ckpt_shape(2, 129, 8) == (2, 2, 8)
