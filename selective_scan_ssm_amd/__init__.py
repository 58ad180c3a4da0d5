"""MI355X (gfx950) selective scan: hand-written HIP kernels behind a C ABI
(include/ssm_scan.h, libssmscan.so) with thin torch wrappers.

    from selective_scan_ssm_amd import scan_fwd, sm1_scan_fwd, state_update

The wrappers are imported lazily so that `selective_scan_ssm_amd.inputs`
(seeded synthetic inputs) can be used without torch or the built library.
"""

__all__ = ["scan_fwd", "sm1_scan_fwd", "state_update", "scan_status", "gated_scan_fwd", "gated_scan_bwd",
           "gated_state_update", "gated_ckpt_shape", "gated_scan_workspace_bytes", "gated_scan_bwd_workspace_bytes",
           "add_rms_norm", "add_rms_norm_quant", "add_rms_norm_bwd", "grad_norm", "clip_grads"]


def __getattr__(name):
    if name in __all__:
        from . import ops
        return getattr(ops, name)
    raise AttributeError(name)
