"""Thin torch-facing wrappers of the C ABI (include/ssm_scan.h).

They only marshal arguments: check devices, dtypes, shapes and contiguity,
allocate outputs (and the workspace) with torch, pass raw device pointers and
torch's current HIP stream to libssmscan.so, and turn a nonzero status into
RuntimeError.  Every step of the computation runs in the library's kernels.
"""
from __future__ import annotations

import array
import operator
from typing import Optional

import torch

from . import _lib

_IO = {torch.float32: _lib.SSM_F32, torch.bfloat16: _lib.SSM_BF16}


def _check(rc: int, what: str):
    if rc != 0:
        raise RuntimeError(f"{what}: {_lib.status_string(rc)}")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _dev(t: torch.Tensor, name: str, dtype=None, shape=None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def scan_fwd(x, delta, A, B, C, D=None, z=None, delta_bias=None, delta_softplus=True, h0=None,
             return_last_state=False, out=None, last_state_out=None, workspace=None, ckpt_out=None):
    """Selective scan.  x, delta, z: (batch, seqlen, d_inner) fp32 or bf16;
    B, C: (batch, seqlen, d_state) same dtype; A: (d_inner, d_state) fp32;
    D, delta_bias: (d_inner,) fp32; h0: (batch, d_inner, d_state) fp32.
    Returns y (same dtype as x) or (y, last_state fp32).  ckpt_out: an fp32
    tensor of ckpt_shape(...) that also receives the state entering every
    16-step block (ssm_scan_fwd_ckpt), for scan_bwd(..., ckpt=ckpt_out)."""
    lib = _lib.load()
    if x.dtype not in _IO:
        raise ValueError("x must be float32 or bfloat16")
    io = x.dtype
    Bt, T, Dd = x.shape
    N = A.shape[-1]
    _dev(x, "x", io)
    _dev(delta, "delta", io, x.shape)
    _dev(z, "z", io, x.shape)
    _dev(B, "B", io, (Bt, T, N))
    _dev(C, "C", io, (Bt, T, N))
    _dev(A, "A", torch.float32, (Dd, N))
    _dev(D, "D", torch.float32, (Dd,))
    _dev(delta_bias, "delta_bias", torch.float32, (Dd,))
    _dev(h0, "h0", torch.float32, (Bt, Dd, N))
    y = out if out is not None else torch.empty_like(x)
    _dev(y, "out", io, x.shape)
    last = None
    if return_last_state:
        last = last_state_out if last_state_out is not None else torch.empty(
            (Bt, Dd, N), dtype=torch.float32, device=x.device)
        _dev(last, "last_state_out", torch.float32, (Bt, Dd, N))
    need = lib.ssm_scan_workspace_bytes(Bt, T, Dd, N, _IO[io])
    if need == (1 << 64) - 1:
        raise RuntimeError("ssm_scan_workspace_bytes: invalid arguments")
    ws = None
    if need:
        ws = workspace if workspace is not None and workspace.numel() >= need else torch.empty(
            need, dtype=torch.uint8, device=x.device)
    if ckpt_out is not None:
        _dev(ckpt_out, "ckpt_out", torch.float32, ckpt_shape(Bt, T, Dd, N))
        rc = lib.ssm_scan_fwd_ckpt(_ptr(x), _ptr(delta), _ptr(delta_bias), int(bool(delta_softplus)),
                                   _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(h0), _ptr(y), _ptr(last),
                                   _ptr(ckpt_out), Bt, T, Dd, N, _IO[io], _ptr(ws), need, _stream(x.device))
        _check(rc, "ssm_scan_fwd_ckpt")
    else:
        rc = lib.ssm_scan_fwd(_ptr(x), _ptr(delta), _ptr(delta_bias), int(bool(delta_softplus)),
                              _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(h0), _ptr(y), _ptr(last),
                              Bt, T, Dd, N, _IO[io], _ptr(ws), need, _stream(x.device))
        _check(rc, "ssm_scan_fwd")
    return (y, last) if return_last_state else y


def ckpt_shape(batch, seqlen, d_inner, d_state):
    """Shape of the saved checkpoints: (batch, ceil(seqlen / 16), d_inner, d_state)."""
    return (batch, (seqlen + 15) // 16, d_inner, d_state)


def sm1_scan_fwd(x, delta, A, B, C, D=None, z=None, delta_bias=None, delta_softplus=True, h0=None,
                 return_last_state=False, out=None, last_state_out=None, workspace=None):
    """d_state = 1 scan.  x, delta, z: (batch, seqlen, d_inner); B, C: (batch, seqlen);
    A, D, delta_bias: (d_inner,); h0, last_state: (batch, d_inner)."""
    lib = _lib.load()
    if x.dtype not in _IO:
        raise ValueError("x must be float32 or bfloat16")
    io = x.dtype
    Bt, T, Dd = x.shape
    _dev(x, "x", io)
    _dev(delta, "delta", io, x.shape)
    _dev(z, "z", io, x.shape)
    _dev(B, "B", io, (Bt, T))
    _dev(C, "C", io, (Bt, T))
    _dev(A, "A", torch.float32, (Dd,))
    _dev(D, "D", torch.float32, (Dd,))
    _dev(delta_bias, "delta_bias", torch.float32, (Dd,))
    _dev(h0, "h0", torch.float32, (Bt, Dd))
    y = out if out is not None else torch.empty_like(x)
    _dev(y, "out", io, x.shape)
    last = None
    if return_last_state:
        last = last_state_out if last_state_out is not None else torch.empty(
            (Bt, Dd), dtype=torch.float32, device=x.device)
        _dev(last, "last_state_out", torch.float32, (Bt, Dd))
    need = lib.sm1_scan_workspace_bytes(Bt, T, Dd, _IO[io])
    if need == (1 << 64) - 1:
        raise RuntimeError("sm1_scan_workspace_bytes: invalid arguments")
    ws = None
    if need:
        ws = workspace if workspace is not None and workspace.numel() >= need else torch.empty(
            need, dtype=torch.uint8, device=x.device)
    rc = lib.sm1_scan_fwd(_ptr(x), _ptr(delta), _ptr(delta_bias), int(bool(delta_softplus)),
                          _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(h0), _ptr(y), _ptr(last),
                          Bt, T, Dd, _IO[io], _ptr(ws), need, _stream(x.device))
    _check(rc, "sm1_scan_fwd")
    return (y, last) if return_last_state else y


def state_update(state, x, delta, A, B, C, D=None, z=None, delta_bias=None, delta_softplus=True,
                 out=None):
    """One decode step; `state` (batch, d_inner, d_state) fp32 is updated in place.
    x, delta, z: (batch, d_inner); B, C: (batch, d_state).  Returns y."""
    lib = _lib.load()
    if x.dtype not in _IO:
        raise ValueError("x must be float32 or bfloat16")
    io = x.dtype
    Bt, Dd = x.shape
    N = A.shape[-1]
    _dev(state, "state", torch.float32, (Bt, Dd, N))
    _dev(x, "x", io)
    _dev(delta, "delta", io, x.shape)
    _dev(z, "z", io, x.shape)
    _dev(B, "B", io, (Bt, N))
    _dev(C, "C", io, (Bt, N))
    _dev(A, "A", torch.float32, (Dd, N))
    _dev(D, "D", torch.float32, (Dd,))
    _dev(delta_bias, "delta_bias", torch.float32, (Dd,))
    y = out if out is not None else torch.empty_like(x)
    _dev(y, "out", io, x.shape)
    rc = lib.ssm_state_update(_ptr(state), _ptr(x), _ptr(delta), _ptr(delta_bias),
                              int(bool(delta_softplus)), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                              _ptr(y), Bt, Dd, N, _IO[io], _stream(x.device))
    _check(rc, "ssm_state_update")
    return y


def scan_bwd(x, delta, A, B, C, dout, D=None, z=None, delta_bias=None, delta_softplus=True,
             h0=None, dlast=None, workspace=None, ckpt=None):
    """Gradient of `scan_fwd`.  Same inputs, plus dout = dL/dy (like x) and
    dlast = dL/dlast_state ((batch, d_inner, d_state) fp32, optional).  Returns
    a dict: dx, ddelta, dB, dC (dtype of x), dA, dh0 (fp32), and dz, dD,
    ddelta_bias (fp32 for dD / ddelta_bias) when z, D, delta_bias are given.
    ckpt: the checkpoints scan_fwd(..., ckpt_out=) recorded on the same inputs
    (ssm_scan_bwd_ckpt); the backward then skips its own checkpoint pass."""
    lib = _lib.load()
    if x.dtype not in _IO:
        raise ValueError("x must be float32 or bfloat16")
    io = x.dtype
    Bt, T, Dd = x.shape
    N = A.shape[-1]
    _dev(x, "x", io)
    _dev(delta, "delta", io, x.shape)
    _dev(z, "z", io, x.shape)
    _dev(dout, "dout", io, x.shape)
    _dev(B, "B", io, (Bt, T, N))
    _dev(C, "C", io, (Bt, T, N))
    _dev(A, "A", torch.float32, (Dd, N))
    _dev(D, "D", torch.float32, (Dd,))
    _dev(delta_bias, "delta_bias", torch.float32, (Dd,))
    _dev(h0, "h0", torch.float32, (Bt, Dd, N))
    _dev(dlast, "dlast", torch.float32, (Bt, Dd, N))
    dev = x.device
    g = dict(dx=torch.empty_like(x), ddelta=torch.empty_like(x), dB=torch.empty_like(B),
             dC=torch.empty_like(C), dA=torch.empty((Dd, N), dtype=torch.float32, device=dev),
             dh0=torch.empty((Bt, Dd, N), dtype=torch.float32, device=dev),
             dz=torch.empty_like(x) if z is not None else None,
             dD=torch.empty((Dd,), dtype=torch.float32, device=dev) if D is not None else None,
             ddelta_bias=torch.empty((Dd,), dtype=torch.float32, device=dev) if delta_bias is not None else None)
    need = lib.ssm_scan_bwd_workspace_bytes(Bt, T, Dd, N, _IO[io])
    if need == (1 << 64) - 1:
        raise RuntimeError("ssm_scan_bwd_workspace_bytes: invalid arguments")
    ws = None
    if need:
        ws = workspace if workspace is not None and workspace.numel() >= need else torch.empty(
            need, dtype=torch.uint8, device=dev)
    outs = (_ptr(g["dx"]), _ptr(g["ddelta"]), _ptr(g["ddelta_bias"]), _ptr(g["dA"]), _ptr(g["dB"]),
            _ptr(g["dC"]), _ptr(g["dD"]), _ptr(g["dz"]), _ptr(g["dh0"]))
    if ckpt is not None:
        _dev(ckpt, "ckpt", torch.float32, ckpt_shape(Bt, T, Dd, N))
        rc = lib.ssm_scan_bwd_ckpt(_ptr(x), _ptr(delta), _ptr(delta_bias), int(bool(delta_softplus)),
                                   _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(h0), _ptr(dout),
                                   _ptr(dlast), _ptr(ckpt), *outs, Bt, T, Dd, N, _IO[io], _ptr(ws), need,
                                   _stream(dev))
        _check(rc, "ssm_scan_bwd_ckpt")
    else:
        rc = lib.ssm_scan_bwd(_ptr(x), _ptr(delta), _ptr(delta_bias), int(bool(delta_softplus)),
                              _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(h0), _ptr(dout),
                              _ptr(dlast), *outs, Bt, T, Dd, N, _IO[io], _ptr(ws), need, _stream(dev))
        _check(rc, "ssm_scan_bwd")
    return g


def dt_proj(xdt, W, out=None):
    """delta = xdt @ W.T, the Mamba block's dt_proj without its bias (the bias
    is the scan's delta_bias).  xdt: (rows, rank) or (batch, seqlen, rank),
    fp32 or bf16, whose last axis is contiguous and whose rows are evenly
    strided: typically the first rank columns of the x_proj output, a view.
    W: (d_inner, rank) in the same dtype.  Returns delta (..., d_inner)."""
    lib = _lib.load()
    if xdt.dtype not in _IO:
        raise ValueError("xdt must be float32 or bfloat16")
    io = xdt.dtype
    if xdt.dim() not in (2, 3) or (xdt.shape[-1] > 1 and xdt.stride(-1) != 1):
        raise ValueError("xdt must be 2-D or 3-D with a contiguous last axis")
    rank = xdt.shape[-1]
    rows = xdt.numel() // rank if rank else 0
    # the stride between consecutive rows, from the leading axes of size > 1
    # (torch may report any stride for an axis of size 1)
    lead = [(n, st) for n, st in zip(xdt.shape[:-1], xdt.stride()[:-1]) if n > 1]
    if len(lead) == 2 and lead[0][1] != lead[1][0] * lead[1][1]:
        raise ValueError("the rows of xdt must be evenly strided")
    ldx = lead[-1][1] if lead else rank
    Dd = W.shape[0]
    if not xdt.is_cuda:
        raise ValueError("xdt must be a GPU tensor")
    _dev(W, "W", io, (Dd, rank))
    y = out if out is not None else torch.empty(tuple(xdt.shape[:-1]) + (Dd,), dtype=io, device=xdt.device)
    _dev(y, "out", io, tuple(xdt.shape[:-1]) + (Dd,))
    rc = lib.ssm_dt_proj(_ptr(xdt), ldx, _ptr(W), _ptr(y), rows, rank, Dd, _IO[io], _stream(xdt.device))
    _check(rc, "ssm_dt_proj")
    return y


def causal_conv1d(x, weight, bias=None, conv_state=None, silu=True, return_state=False, out=None):
    """Causal depthwise conv1d (+ SiLU) of the Mamba block's x branch.
    x: (batch, seqlen, d_inner) fp32 or bf16; weight: (d_inner, width) fp32;
    bias: (d_inner,) fp32; conv_state: (batch, d_inner, width - 1) like x, the
    inputs before the sequence.  Returns out, or (out, new conv_state)."""
    lib = _lib.load()
    if x.dtype not in _IO:
        raise ValueError("x must be float32 or bfloat16")
    io = x.dtype
    Bt, T, Dd = x.shape
    K = weight.shape[-1]
    _dev(x, "x", io)
    _dev(weight, "weight", torch.float32, (Dd, K))
    _dev(bias, "bias", torch.float32, (Dd,))
    _dev(conv_state, "conv_state", io, (Bt, Dd, K - 1))
    y = out if out is not None else torch.empty_like(x)
    _dev(y, "out", io, x.shape)
    st = torch.empty((Bt, Dd, K - 1), dtype=io, device=x.device) if return_state else None
    rc = lib.ssm_causal_conv1d_fwd(_ptr(x), _ptr(weight), _ptr(bias), _ptr(conv_state), _ptr(y),
                                   _ptr(st), int(bool(silu)), Bt, T, Dd, K, _IO[io], _stream(x.device))
    _check(rc, "ssm_causal_conv1d_fwd")
    return (y, st) if return_state else y


def causal_conv1d_update(conv_state, x, weight, bias=None, silu=True, out=None):
    """One decode token: conv_state (batch, d_inner, width - 1) is updated in
    place; x: (batch, d_inner).  Returns out (batch, d_inner)."""
    lib = _lib.load()
    if x.dtype not in _IO:
        raise ValueError("x must be float32 or bfloat16")
    io = x.dtype
    Bt, Dd = x.shape
    K = weight.shape[-1]
    _dev(conv_state, "conv_state", io, (Bt, Dd, K - 1))
    _dev(x, "x", io)
    _dev(weight, "weight", torch.float32, (Dd, K))
    _dev(bias, "bias", torch.float32, (Dd,))
    y = out if out is not None else torch.empty_like(x)
    _dev(y, "out", io, x.shape)
    rc = lib.ssm_causal_conv1d_update(_ptr(conv_state), _ptr(x), _ptr(weight), _ptr(bias), _ptr(y),
                                      int(bool(silu)), Bt, Dd, K, _IO[io], _stream(x.device))
    _check(rc, "ssm_causal_conv1d_update")
    return y


def scan_fwd_2d(x, delta, A, B, C, height, width, direction, D=None, z=None, delta_bias=None,
                delta_softplus=True, h0=None, return_last_state=False, out=None, workspace=None):
    """One direction (0 row-major, 1 reverse, 2 column-major, 3 reverse
    column-major) of the 2-D scan over height x width patches held row-major
    on the sequence axis; y comes back at each patch's position."""
    lib = _lib.load()
    if x.dtype not in _IO:
        raise ValueError("x must be float32 or bfloat16")
    io = x.dtype
    Bt, T, Dd = x.shape
    N = A.shape[-1]
    if T != height * width:
        raise ValueError("seqlen must be height * width")
    _dev(x, "x", io)
    _dev(delta, "delta", io, x.shape)
    _dev(z, "z", io, x.shape)
    _dev(B, "B", io, (Bt, T, N))
    _dev(C, "C", io, (Bt, T, N))
    _dev(A, "A", torch.float32, (Dd, N))
    _dev(D, "D", torch.float32, (Dd,))
    _dev(delta_bias, "delta_bias", torch.float32, (Dd,))
    _dev(h0, "h0", torch.float32, (Bt, Dd, N))
    y = out if out is not None else torch.empty_like(x)
    _dev(y, "out", io, x.shape)
    last = torch.empty((Bt, Dd, N), dtype=torch.float32, device=x.device) if return_last_state else None
    need = lib.ssm_scan_2d_workspace_bytes(Bt, height, width, Dd, N, int(direction), int(z is not None), _IO[io])
    if need == (1 << 64) - 1:
        raise RuntimeError("ssm_scan_2d_workspace_bytes: invalid arguments")
    ws = None
    if need:
        ws = workspace if workspace is not None and workspace.numel() >= need else torch.empty(
            need, dtype=torch.uint8, device=x.device)
    rc = lib.ssm_scan_fwd_2d(_ptr(x), _ptr(delta), _ptr(delta_bias), int(bool(delta_softplus)),
                             _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(h0), _ptr(y), _ptr(last),
                             Bt, height, width, Dd, N, int(direction), _IO[io], _ptr(ws), need,
                             _stream(x.device))
    _check(rc, "ssm_scan_fwd_2d")
    return (y, last) if return_last_state else y


def ssd_scan_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=True, h0=None,
                 return_last_state=False, out=None, last_state_out=None, workspace=None):
    """Mamba-2 multi-head scan.  x, z: (batch, seqlen, nheads, headdim) fp32 or
    bf16; dt: (batch, seqlen, nheads); B, C: (batch, seqlen, dstate) same dtype;
    A, D, dt_bias: (nheads,) fp32; h0: (batch, nheads, headdim, dstate) fp32.
    Returns y (same dtype as x) or (y, last_state fp32)."""
    lib = _lib.load()
    if x.dtype not in _IO:
        raise ValueError("x must be float32 or bfloat16")
    io = x.dtype
    Bt, T, H, P = x.shape
    N = B.shape[-1]
    _dev(x, "x", io)
    _dev(dt, "dt", io, (Bt, T, H))
    _dev(z, "z", io, x.shape)
    _dev(B, "B", io, (Bt, T, N))
    _dev(C, "C", io, (Bt, T, N))
    _dev(A, "A", torch.float32, (H,))
    _dev(D, "D", torch.float32, (H,))
    _dev(dt_bias, "dt_bias", torch.float32, (H,))
    _dev(h0, "h0", torch.float32, (Bt, H, P, N))
    y = out if out is not None else torch.empty_like(x)
    _dev(y, "out", io, x.shape)
    last = None
    if return_last_state:
        last = last_state_out if last_state_out is not None else torch.empty(
            (Bt, H, P, N), dtype=torch.float32, device=x.device)
        _dev(last, "last_state_out", torch.float32, (Bt, H, P, N))
    need = lib.ssd_scan_workspace_bytes(Bt, T, H, P, N, _IO[io])
    if need == (1 << 64) - 1:
        raise RuntimeError("ssd_scan_workspace_bytes: invalid arguments")
    ws = None
    if need:
        ws = workspace if workspace is not None and workspace.numel() >= need else torch.empty(
            need, dtype=torch.uint8, device=x.device)
    rc = lib.ssd_scan_fwd(_ptr(x), _ptr(dt), _ptr(dt_bias), int(bool(dt_softplus)), _ptr(A), _ptr(B),
                          _ptr(C), _ptr(D), _ptr(z), _ptr(h0), _ptr(y), _ptr(last), Bt, T, H, P, N,
                          _IO[io], _ptr(ws), need, _stream(x.device))
    _check(rc, "ssd_scan_fwd")
    return (y, last) if return_last_state else y


def scan_status(workspace, stream_device=None):
    """ssm_scan_status on a workspace tensor (uint8, device) of the last
    forward scan: 0 (SSM_OK) or SSM_ERR_WAIT when a segment's bounded wait
    gave up.  Synchronises torch's current stream of the workspace's device."""
    lib = _lib.load()
    dev = workspace.device if stream_device is None else stream_device
    return lib.ssm_scan_status(_ptr(workspace), workspace.numel(), _stream(dev))


def scan_workspace_bytes(batch, seqlen, d_inner, d_state, dtype):
    """ssm_scan_workspace_bytes for io dtype `dtype` (torch.float32 / torch.bfloat16)."""
    need = _lib.load().ssm_scan_workspace_bytes(batch, seqlen, d_inner, d_state, _IO[dtype])
    if need == (1 << 64) - 1:
        raise RuntimeError("ssm_scan_workspace_bytes: invalid arguments")
    return need


def conv_scan_fwd(x, conv_weight, delta, A, B, C, conv_bias=None, conv_state=None, D=None, z=None,
                  delta_bias=None, delta_softplus=True, h0=None, return_last_state=False,
                  return_conv_state=False, out=None, workspace=None):
    """The block's prologue and the scan in one call (ssm_conv_scan_fwd): the
    scan of scan_fwd on SiLU(causal_conv1d(x)).  x: (batch, seqlen, d_inner)
    conv input; conv_weight: (d_inner, width) fp32; conv_bias: (d_inner,)
    fp32; conv_state: (batch, d_inner, width - 1) in x's dtype.  Returns y,
    plus last_state and/or the conv window after the sequence when asked."""
    lib = _lib.load()
    if x.dtype not in _IO:
        raise ValueError("x must be float32 or bfloat16")
    io = x.dtype
    Bt, T, Dd = x.shape
    N = A.shape[-1]
    K = conv_weight.shape[-1]
    _dev(x, "x", io)
    _dev(conv_weight, "conv_weight", torch.float32, (Dd, K))
    _dev(conv_bias, "conv_bias", torch.float32, (Dd,))
    _dev(conv_state, "conv_state", io, (Bt, Dd, K - 1))
    _dev(delta, "delta", io, x.shape)
    _dev(z, "z", io, x.shape)
    _dev(B, "B", io, (Bt, T, N))
    _dev(C, "C", io, (Bt, T, N))
    _dev(A, "A", torch.float32, (Dd, N))
    _dev(D, "D", torch.float32, (Dd,))
    _dev(delta_bias, "delta_bias", torch.float32, (Dd,))
    _dev(h0, "h0", torch.float32, (Bt, Dd, N))
    y = out if out is not None else torch.empty_like(x)
    _dev(y, "out", io, x.shape)
    last = torch.empty((Bt, Dd, N), dtype=torch.float32, device=x.device) if return_last_state else None
    win = torch.empty((Bt, Dd, K - 1), dtype=io, device=x.device) if return_conv_state else None
    need = lib.ssm_conv_scan_workspace_bytes(Bt, T, Dd, N, _IO[io])
    if need == (1 << 64) - 1:
        raise RuntimeError("ssm_conv_scan_workspace_bytes: invalid arguments")
    ws = None
    if need:
        ws = workspace if workspace is not None and workspace.numel() >= need else torch.empty(
            need, dtype=torch.uint8, device=x.device)
    rc = lib.ssm_conv_scan_fwd(_ptr(x), _ptr(conv_weight), _ptr(conv_bias), _ptr(conv_state), _ptr(win), K,
                               _ptr(delta), _ptr(delta_bias), int(bool(delta_softplus)), _ptr(A), _ptr(B),
                               _ptr(C), _ptr(D), _ptr(z), _ptr(h0), _ptr(y), _ptr(last), Bt, T, Dd, N, _IO[io],
                               _ptr(ws), need, _stream(x.device))
    _check(rc, "ssm_conv_scan_fwd")
    res = (y,)
    if return_last_state:
        res += (last,)
    if return_conv_state:
        res += (win,)
    return res if len(res) > 1 else y


# ------------------------------------------------- the gated recurrent block
# A decode step's kernels run for a few microseconds, so these wrappers check
# each tensor with one test that passes (its message is put together only when
# it fails) and take the stream handle without building a Stream object.
_raw_stream = torch._C._cuda_getCurrentRawStream
_BAD = (1 << 64) - 1


def _device(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    return t.device


def _arg(t, name, dtype, shape, dev):
    """The address of a contiguous tensor of this dtype and shape on dev (None for None)."""
    if t is None:
        return None
    if t.dtype != dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        _dev(t, name, dtype, shape)
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    return t.data_ptr()


def _out(t, name, like, dtype, shape, dev):
    """The caller's output tensor, or a new one of like's shape; and its address."""
    if t is not None:
        return t, _arg(t, name, dtype, shape, dev)
    # empty_like is the cheapest allocation, but keeps a strided tensor's gaps
    t = torch.empty_like(like, dtype=dtype) if like.is_contiguous() else torch.empty(shape, dtype=dtype, device=dev)
    return t, t.data_ptr()


def _rows(t, name, dtype, shape, dev):
    """The address of t and the stride between its consecutive rows: its last
    axis is contiguous and its other axes step evenly (a column range of a
    wider tensor)."""
    if t is None:
        return None, 0
    if t.dtype == dtype and t.shape == shape and t.device == dev and t.is_contiguous():
        return t.data_ptr(), shape[-1]
    _device(t, name)
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    dim = shape[-1]
    if dim > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have a contiguous last axis")
    lead = [(n, st) for n, st in zip(t.shape[:-1], t.stride()[:-1]) if n > 1]
    for (_, outer), (n, inner) in zip(lead, lead[1:]):
        if outer != n * inner:
            raise ValueError(f"the rows of {name} must be evenly strided")
    ld = lead[-1][1] if lead else dim
    if ld < dim:
        raise ValueError(f"the rows of {name} overlap")
    return t.data_ptr(), ld


def _run(dev, fn, *args):
    """fn(*args, stream) with dev as the current device, on its current stream."""
    index = dev.index
    if torch.cuda.current_device() == index:
        return fn(*args, _raw_stream(index))
    with torch.cuda.device(dev):
        return fn(*args, _raw_stream(index))


def _scratch(need, what, workspace, dev, status=False):
    """A workspace of `need` bytes: the caller's if it is large enough.  Returns
    it (the caller holds it until the launch) and its address.  status: the call
    leaves an error word that scan_status reads in the caller's workspace, so a
    smaller one is refused and not replaced."""
    if need == _BAD:
        raise RuntimeError(f"{what}: invalid arguments")
    if not need:
        return None, None
    if status and workspace is not None and workspace.numel() < need:
        raise ValueError(f"workspace holds {workspace.numel()} bytes, {need} are needed")
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    return workspace, _arg(workspace, "workspace", torch.uint8, workspace.shape, dev)


def gated_ckpt_shape(batch, seqlen, d_inner):
    """Shape of gated_scan_fwd's checkpoints: (batch, ceil(seqlen / 128), d_inner)."""
    return (batch, -(-seqlen // _lib.GATED_BLOCK), d_inner)


def gated_scan_workspace_bytes(batch, seqlen, d_inner, dtype):
    """Bytes of gated_scan_fwd's workspace (0 up to 128 steps)."""
    return _gated_bytes(_lib.load().ssm_gated_scan_workspace_bytes, batch, seqlen, d_inner, dtype)


def gated_scan_bwd_workspace_bytes(batch, seqlen, d_inner, dtype):
    """Bytes of gated_scan_bwd's workspace, with or without ckpt."""
    return _gated_bytes(_lib.load().ssm_gated_scan_bwd_workspace_bytes, batch, seqlen, d_inner, dtype)


def _gated_bytes(fn, batch, seqlen, d_inner, dtype):
    need = fn(batch, seqlen, d_inner, _IO[dtype])
    if need == _BAD:
        raise RuntimeError(f"{fn.__name__}: invalid arguments")
    return need


def gated_scan_fwd(x, g, z=None, gate_bias=None, h0=None, return_last_state=False, out=None, last_state_out=None,
                   ckpt_out=None, workspace=None):
    """Gated linear recurrence: a = sigmoid(g + gate_bias), h <- a h + (1 - a) x,
    y = h SiLU(z) (y = h without z).  x, g, z: (batch, seqlen, d_inner) fp32 or
    bf16 with a contiguous last axis and evenly strided rows (thirds of one
    projection's output need no copy); gate_bias: (d_inner,) fp32; h0: (batch,
    d_inner) fp32.  g = +inf keeps the state, g = -inf restarts it (x finite at
    such a step, and the state that a restart leaves behind).  Returns y
    (same dtype as x) or (y, last_state fp32).  ckpt_out: an fp32 tensor of
    gated_ckpt_shape(...) that also receives the state entering every 128-step
    block, for gated_scan_bwd(..., ckpt=ckpt_out).  workspace: a uint8 tensor of at
    least gated_scan_workspace_bytes(...), allocated here without one; scan_status
    reads the call's outcome in it (nothing is written up to 128 steps, which need none)."""
    lib = _lib.load()
    io, dev, shape = x.dtype, _device(x, "x"), x.shape
    if io not in _IO:
        raise ValueError("x must be float32 or bfloat16")
    Bt, T, Dd = shape
    px, ldx = _rows(x, "x", io, shape, dev)
    pg, ldg = _rows(g, "g", io, shape, dev)
    pz, ldz = _rows(z, "z", io, shape, dev)
    y, py = _out(out, "out", x, io, shape, dev)
    last = None
    if return_last_state:
        last = last_state_out if last_state_out is not None else torch.empty((Bt, Dd), dtype=torch.float32, device=dev)
    ws, pws = _scratch(lib.ssm_gated_scan_workspace_bytes(Bt, T, Dd, _IO[io]), "ssm_gated_scan_workspace_bytes",
                       workspace, dev, status=True)
    rc = _run(dev, lib.ssm_gated_scan_fwd, px, ldx, pg, ldg, _arg(gate_bias, "gate_bias", torch.float32, (Dd,), dev), pz,
              ldz, _arg(h0, "h0", torch.float32, (Bt, Dd), dev), py,
              _arg(last, "last_state_out", torch.float32, (Bt, Dd), dev),
              _arg(ckpt_out, "ckpt_out", torch.float32, gated_ckpt_shape(Bt, T, Dd), dev), Bt, T, Dd, _IO[io], pws,
              0 if ws is None else ws.numel())
    _check(rc, "ssm_gated_scan_fwd")
    return (y, last) if return_last_state else y


def gated_scan_bwd(x, g, dout, z=None, gate_bias=None, h0=None, dlast=None, ckpt=None, workspace=None):
    """Gradient of gated_scan_fwd.  Same inputs, plus dout = dL/dy (contiguous,
    like y) and dlast = dL/dlast_state ((batch, d_inner) fp32, optional).
    Returns a dict: dx, dg (dtype of x), dh0 (fp32), and dz, dgate_bias (fp32)
    when z, gate_bias are given (None otherwise).  ckpt: what
    gated_scan_fwd(..., ckpt_out=) recorded on the same inputs; without it the
    call reads x and g once more.  workspace: as in gated_scan_fwd, of at least
    gated_scan_bwd_workspace_bytes(...)."""
    lib = _lib.load()
    io, dev, shape = x.dtype, _device(x, "x"), x.shape
    if io not in _IO:
        raise ValueError("x must be float32 or bfloat16")
    Bt, T, Dd = shape
    px, ldx = _rows(x, "x", io, shape, dev)
    pg, ldg = _rows(g, "g", io, shape, dev)
    pz, ldz = _rows(z, "z", io, shape, dev)
    new = lambda size, dtype: torch.empty(size, dtype=dtype, device=dev)
    dx, dg, dz = new(shape, io), new(shape, io), new(shape, io) if z is not None else None
    dbias = new((Dd,), torch.float32) if gate_bias is not None else None
    dh0 = new((Bt, Dd), torch.float32)
    ws, pws = _scratch(lib.ssm_gated_scan_bwd_workspace_bytes(Bt, T, Dd, _IO[io]), "ssm_gated_scan_bwd_workspace_bytes",
                       workspace, dev, status=True)
    rc = _run(dev, lib.ssm_gated_scan_bwd, px, ldx, pg, ldg, _arg(gate_bias, "gate_bias", torch.float32, (Dd,), dev), pz,
              ldz, _arg(h0, "h0", torch.float32, (Bt, Dd), dev), _arg(dout, "dout", io, shape, dev),
              _arg(dlast, "dlast", torch.float32, (Bt, Dd), dev),
              _arg(ckpt, "ckpt", torch.float32, gated_ckpt_shape(Bt, T, Dd), dev), _ptr(dx), _ptr(dg), _ptr(dz),
              _ptr(dbias), _ptr(dh0), Bt, T, Dd, _IO[io], pws, 0 if ws is None else ws.numel())
    _check(rc, "ssm_gated_scan_bwd")
    return dict(dx=dx, dg=dg, dz=dz, dgate_bias=dbias, dh0=dh0)


def gated_state_update(state, x, g, z=None, gate_bias=None, out=None):
    """One decode token of gated_scan_fwd; `state` (batch, d_inner) fp32 is
    updated in place.  x, g, z: (batch, d_inner).  Returns y."""
    lib = _lib.load()
    io, dev, shape = x.dtype, _device(x, "x"), x.shape
    if io not in _IO:
        raise ValueError("x must be float32 or bfloat16")
    Bt, Dd = shape
    px = _arg(x, "x", io, shape, dev)
    y, py = _out(out, "out", x, io, shape, dev)
    rc = _run(dev, lib.ssm_gated_state_update, _arg(state, "state", torch.float32, shape, dev), px,
              _arg(g, "g", io, shape, dev), _arg(gate_bias, "gate_bias", torch.float32, (Dd,), dev),
              _arg(z, "z", io, shape, dev), py, Bt, Dd, _IO[io])
    _check(rc, "ssm_gated_state_update")
    return y


def _norm_residual(x, io, residual, residual_dtype, residual_out, dev):
    """The residual's dtype and address, the tensor that r goes to (None: r is x
    itself) and its address."""
    if residual is not None:
        if residual_dtype is not None and residual_dtype != residual.dtype:
            raise ValueError("residual_dtype differs from residual's dtype")
        res = residual.dtype
    elif residual_dtype is not None:
        res = residual_dtype
    else:
        res = residual_out.dtype if residual_out is not None else io
    if res != io and res != torch.float32:
        raise ValueError(f"the residual must be float32 or {io}, got {res}")
    shape = x.shape
    pr = _arg(residual, "residual", res, shape, dev)
    if residual is None and residual_dtype is None and residual_out is None:
        return res, None, None, None
    r, po = _out(residual_out, "residual_out", x if residual is None else residual, res, shape, dev)
    return res, pr, r, po


def add_rms_norm(x, weight, residual=None, eps=1e-5, residual_dtype=None, out=None, residual_out=None):
    """r = x + residual, y = r / sqrt(mean(r^2) + eps) * weight over the last
    axis.  x: (..., dim) fp32 or bf16, rows evenly strided; weight: (dim,) fp32;
    residual: x's shape, contiguous, in x's dtype or fp32.  Returns (y, r): y in x's dtype, r
    in the residual's (residual_dtype when there is no residual; without either
    r is None, as it would be x itself).  residual_out may be residual, which is
    then updated in place."""
    lib = _lib.load()
    io, dev, shape = x.dtype, _device(x, "x"), x.shape
    if io not in _IO or not shape:
        raise ValueError("x must be float32 or bfloat16, with at least one axis")
    dim = shape[-1]
    px, ldx = _rows(x, "x", io, shape, dev)
    res, pr, r, po = _norm_residual(x, io, residual, residual_dtype, residual_out, dev)
    y, py = _out(out, "out", x, io, shape, dev)
    rc = _run(dev, lib.ssm_add_rms_norm_fwd, px, ldx, pr, _arg(weight, "weight", torch.float32, (dim,), dev), py, po,
              x.numel() // dim if dim else 0, dim, eps, _IO[io], _IO[res])
    _check(rc, "ssm_add_rms_norm_fwd")
    return y, r


def add_rms_norm_quant(x, weight, residual=None, eps=1e-5, residual_dtype=None, out=None, scale_out=None,
                       residual_out=None):
    """add_rms_norm with an 8-bit output: returns (q, scale, r), q in
    float8_e4m3fn and scale (x.shape[:-1]) fp32 with q * scale standing for y,
    scale = max(max |y| / 448, 2^-126) per row."""
    lib = _lib.load()
    io, dev, shape = x.dtype, _device(x, "x"), x.shape
    if io not in _IO or not shape:
        raise ValueError("x must be float32 or bfloat16, with at least one axis")
    dim = shape[-1]
    px, ldx = _rows(x, "x", io, shape, dev)
    res, pr, r, po = _norm_residual(x, io, residual, residual_dtype, residual_out, dev)
    q, pq = _out(out, "out", x, torch.float8_e4m3fn, shape, dev)
    scale = scale_out if scale_out is not None else torch.empty(shape[:-1], dtype=torch.float32, device=dev)
    rc = _run(dev, lib.ssm_add_rms_norm_quant, px, ldx, pr, _arg(weight, "weight", torch.float32, (dim,), dev), pq,
              _arg(scale, "scale_out", torch.float32, shape[:-1], dev), po, x.numel() // dim if dim else 0, dim, eps,
              _IO[io], _IO[res])
    _check(rc, "ssm_add_rms_norm_quant")
    return q, scale, r


def add_rms_norm_bwd(dy, r, weight, dresidual=None, eps=1e-5, dresidual_out=None, workspace=None):
    """Gradient of add_rms_norm at the r it returned (x itself when it returned
    None).  dy: dL/dy (..., dim) fp32 or bf16, contiguous; r: like dy, in its
    dtype or fp32, rows evenly strided (an x that the forward took so);
    dresidual: dL/dr from the residual stream, r's dtype, contiguous, optional.  Returns a
    dict: dx (dy's dtype), dresidual (the gradient of residual: dx itself when
    the dtypes are the same, else in r's dtype) and dweight (dim,) fp32.
    dresidual_out: where dresidual goes, may be dresidual itself."""
    lib = _lib.load()
    io, dev, shape, res = dy.dtype, _device(dy, "dy"), dy.shape, r.dtype
    if io not in _IO or not shape:
        raise ValueError("dy must be float32 or bfloat16, with at least one axis")
    if res != io and res != torch.float32:
        raise ValueError(f"r must be float32 or {io}, got {res}")
    dim = shape[-1]
    rows = dy.numel() // dim if dim else 0
    pdy = _arg(dy, "dy", io, shape, dev)
    pr, ldr = _rows(r, "r", res, shape, dev)
    dx = torch.empty_like(dy)
    own = dresidual_out if dresidual_out is not None else (torch.empty(shape, dtype=res, device=dev) if res != io else None)
    dw = torch.empty((dim,), dtype=torch.float32, device=dev)
    ws, pws = _scratch(lib.ssm_add_rms_norm_bwd_workspace_bytes(rows, dim), "ssm_add_rms_norm_bwd_workspace_bytes",
                       workspace, dev)
    rc = _run(dev, lib.ssm_add_rms_norm_bwd_strided, pdy, pr, ldr,
              _arg(weight, "weight", torch.float32, (dim,), dev), _arg(dresidual, "dresidual", res, shape, dev), _ptr(dx),
              _arg(own, "dresidual_out", res, shape, dev), _ptr(dw), rows, dim, eps, _IO[io], _IO[res], pws,
              0 if ws is None else ws.numel())
    _check(rc, "ssm_add_rms_norm_bwd_strided")
    return dict(dx=dx, dresidual=dx if own is None else own, dweight=dw)


_dtype_of = operator.attrgetter("dtype")


def _grad_list(tensors, name, dev):
    """Host arrays (addresses, dtypes) of a list of contiguous tensors on dev.
    A few hundred tensors cost more here than on the GPU, so every attribute is
    read in one C-level pass."""
    kinds = set(map(_dtype_of, tensors))
    if not kinds <= _IO.keys():
        raise ValueError(f"{name} must be float32 or bfloat16, got {kinds}")
    # get_device() is -1 for a CPU tensor
    if set(map(torch.Tensor.get_device, tensors)) != {dev.index}:
        raise ValueError(f"{name} must all be on {dev}")
    if not all(map(torch.Tensor.is_contiguous, tensors)):
        raise ValueError(f"{name} must be contiguous")
    if len(kinds) == 1:
        codes = array.array("i", (_IO[kinds.pop()],)) * len(tensors)
    else:
        codes = array.array("i", map(_IO.__getitem__, map(_dtype_of, tensors)))
    return array.array("Q", map(torch.Tensor.data_ptr, tensors)), codes


def _at(host):
    """The address of a host array."""
    return host.buffer_info()[0]


def _clip(grads, max_norm, out, eps, norm_out, workspace):
    lib = _lib.load()
    grads = list(grads)
    if not grads:
        raise ValueError("the list of gradients is empty")
    dev = _device(grads[0], "every gradient")
    n = len(grads)
    ptrs, dtypes = _grad_list(grads, "gradients", dev)
    sizes = list(map(torch.Tensor.numel, grads))
    numel = array.array("q", sizes)
    norm = norm_out if norm_out is not None else torch.empty((), dtype=torch.float32, device=dev)
    if norm.numel() != 1:
        raise ValueError("norm_out must hold one value")
    pn = _arg(norm, "norm_out", torch.float32, norm.shape, dev)
    ws, pws = _scratch(lib.ssm_grad_norm_workspace_bytes(n), "ssm_grad_norm_workspace_bytes", workspace, dev)
    if max_norm is None:
        rc = _run(dev, lib.ssm_grad_norm, _at(ptrs), _at(numel), _at(dtypes), n, pn, pws, ws.numel())
        _check(rc, "ssm_grad_norm")
        return norm
    outs = out_dtypes = None
    if out is not None:
        out = list(out)
        if list(map(torch.Tensor.numel, out)) != sizes:
            raise ValueError("out must have the gradients' sizes")
        outs, out_dtypes = _grad_list(out, "out", dev)
    rc = _run(dev, lib.ssm_grad_clip, _at(ptrs), None if outs is None else _at(outs), _at(numel), _at(dtypes),
              None if outs is None else _at(out_dtypes), n, max_norm, eps, pn, pws, ws.numel())
    _check(rc, "ssm_grad_clip")
    return norm


def grad_norm(grads, norm_out=None, workspace=None):
    """sqrt(sum of squares) over a list of contiguous fp32 / bf16 tensors, as
    an fp32 scalar on their device."""
    return _clip(grads, None, None, 0.0, norm_out, workspace)


def clip_grads(grads, max_norm, out=None, eps=1e-6, norm_out=None, workspace=None):
    """Scales a list of contiguous fp32 / bf16 tensors by min(1, max_norm /
    (norm + eps)), norm being grad_norm(grads): in place, or into the tensors
    of `out` (same numbers of elements, fp32 or bf16 each: an optimizer's fp32 gradients
    from bf16 ones).  An infinite max_norm is no limit.  Returns the norm before clipping.  The host never waits."""
    if max_norm is None:
        raise ValueError("max_norm must be a number")
    return _clip(grads, float(max_norm), out, float(eps), norm_out, workspace)
