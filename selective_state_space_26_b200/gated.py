"""The gated linear recurrence: binding of include/jamba_ssm_gated.h.

    u_t = rate * sigmoid(g_t + bias),  h_t = h_{t-1} + u_t (x_t - h_{t-1}),
    out_t = h_t * silu(z_t)

with one state per channel.  Every step runs in the kernels of
libjamba_ssm_gated.so; this module checks tensor metadata, allocates outputs
and hands over pointers and the stream.
"""
from __future__ import annotations

from ctypes import byref, sizeof

import torch

from . import _lib
from ._lib import JambaSSMError
from ._tensors import (IO, check, cuda_device, empty_like, launching, need, ptr,
                       raw_stream, row_stride, status_device)
from ._tensors import workspace as _workspace

__all__ = ["jamba_ssm_gated_scan", "jamba_ssm_gated_scan_ckpt", "jamba_ssm_gated_scan_ckpt_size",
           "jamba_ssm_gated_scan_bwd", "jamba_ssm_gated_scan_bwd_workspace_size",
           "jamba_ssm_gated_state_update", "jamba_ssm_gated_get_status"]

_F32, _I32 = torch.float32, torch.int32
_SCAN, _BWD, _UPDATE = (sizeof(c) for c in (_lib.GatedScanParams, _lib.GatedScanBwdParams,
                                            _lib.GatedStateUpdateParams))


def _raise(status, what):
    raise JambaSSMError(status, what, cuda_error=_lib.gated_lib().jamba_ssm_gated_last_cuda_error())


def _sizes(x, cu_seqlens, dev):
    """(batch, seqlen, rows, d_inner) of batched or packed activations."""
    if x.dtype not in IO:
        raise TypeError(f"x must be bfloat16 or float32, got {x.dtype}")
    if cu_seqlens is None:
        if x.dim() != 3:
            raise ValueError(f"x must be [batch, seqlen, d_inner], got {tuple(x.shape)}")
        batch, seqlen, d = x.shape
        return batch, seqlen, batch * seqlen, d
    if x.dim() != 2:
        raise ValueError(f"packed x must be [tokens, d_inner], got {tuple(x.shape)}")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be [batch + 1]")
    check(cu_seqlens, "cu_seqlens", cu_seqlens.shape, _I32, dev)
    return cu_seqlens.numel() - 1, 0, x.shape[0], x.shape[1]


def jamba_ssm_gated_scan(x, g, z=None, rate=None, bias=None, h0=None, out=None, h_final=None,
                         return_final_state=True, cu_seqlens=None, state_indices=None,
                         initial_indices=None, ckpt=None, workspace=None, stream=None):
    """Scan over whole sequences.  x, g and (optionally) z [batch, seqlen,
    d_inner] bf16 or fp32, whose rows may be evenly strided (column blocks of
    one projection's output); rate (in [0, 1]) and bias [d_inner] fp32 or None;
    h0 [batch, d_inner] fp32 or None.  Returns (out, h_final); h_final is None
    when return_final_state is False and no buffer was passed.

    With ``cu_seqlens`` (int32 [batch + 1]) the activations are packed [tokens,
    d_inner] and sequence b is rows cu_seqlens[b]:cu_seqlens[b+1].  With
    ``state_indices`` (int32 [batch]) h0 / h_final are [num_slots, d_inner]
    caches: sequence b's final state goes to row state_indices[b] (negative: not
    written), its initial state comes from row initial_indices[b] (None:
    state_indices[b]; negative: zero); pass h_final explicitly then.

    ``ckpt``: a buffer of ``jamba_ssm_gated_scan_ckpt`` that receives what
    ``jamba_ssm_gated_scan_bwd`` on the same inputs can take.  ``workspace``: an
    optional zero-filled tensor of 16 bytes that holds this call's status word."""
    dev = cuda_device(x, "x", "jamba_ssm_gated_scan")
    batch, seqlen, rows, d = _sizes(x, cu_seqlens, dev)
    io, shape = x.dtype, x.shape
    xs = row_stride(x, "x", shape, io, dev)
    gs = row_stride(g, "g", shape, io, dev, required=True)
    zs = row_stride(z, "z", shape, io, dev)
    check(rate, "rate", (d,), _F32, dev)
    check(bias, "bias", (d,), _F32, dev)
    slots = 0
    if initial_indices is not None and state_indices is None:
        raise ValueError("initial_indices needs state_indices")
    if state_indices is not None:
        check(state_indices, "state_indices", (batch,), _I32, dev)
        check(initial_indices, "initial_indices", (batch,), _I32, dev)
        if h0 is None and h_final is None:
            raise ValueError("state_indices needs a cache: h0, h_final or both")
        slots = (h_final if h0 is None else h0).shape[0]
    state = (batch if state_indices is None else slots, d)
    check(h0, "h0", state, _F32, dev)
    check(h_final, "h_final", state, _F32, dev)
    check(out, "out", shape, io, dev)
    if ckpt is not None:
        check(ckpt, "ckpt", (rows // _lib.GATED_CKPT_STEPS + batch, d), _F32, dev)
    ws, ws_bytes = _workspace(workspace, dev)
    with launching(stream, dev):
        if out is None:
            out = empty_like(x, xs == 0)
        if h_final is None and return_final_state and state_indices is None:
            h_final = x.new_empty(state, dtype=_F32) if h0 is None else empty_like(h0)
        p = _lib.GatedScanParams(_SCAN, batch, seqlen, d, IO[io], 0, x.data_ptr(), g.data_ptr(),
                                 ptr(z), xs, gs, zs, ptr(rate), ptr(bias), ptr(h0), ptr(out), ptr(h_final),
                                 ptr(cu_seqlens), rows, ptr(state_indices), ptr(initial_indices),
                                 slots, ptr(ckpt), ws, ws_bytes)
        st = _lib.gated_lib().jamba_ssm_gated_scan(byref(p), raw_stream(dev))
    if st != _lib.OK:
        _raise(st, "jamba_ssm_gated_scan")
    return out, h_final


def jamba_ssm_gated_scan_ckpt(x, cu_seqlens=None):
    """An empty checkpoint buffer for a scan of x (fp32 [entries, d_inner])."""
    if cu_seqlens is None:
        batch, rows = x.shape[0], x.shape[0] * x.shape[1]
    else:
        batch, rows = cu_seqlens.numel() - 1, x.shape[0]
    return torch.empty(rows // _lib.GATED_CKPT_STEPS + batch, x.shape[-1], dtype=_F32,
                       device=x.device)


def jamba_ssm_gated_scan_ckpt_size(batch: int, rows: int, d_inner: int) -> int:
    """Bytes of the checkpoints of `batch` sequences of `rows` tokens in all."""
    return _lib.gated_lib().jamba_ssm_gated_scan_ckpt_size(int(batch), int(rows), int(d_inner))


def jamba_ssm_gated_scan_bwd_workspace_size(batch: int, rows: int, d_inner: int,
                                            has_ckpt: bool = False) -> int:
    """Bytes of the workspace the backward pass needs."""
    return _lib.gated_lib().jamba_ssm_gated_scan_bwd_workspace_size(int(batch), int(rows),
                                                                    int(d_inner), int(has_ckpt))


def jamba_ssm_gated_scan_bwd(x, g, dout, z=None, rate=None, bias=None, h0=None, dh_final=None,
                             cu_seqlens=None, ckpt=None, workspace=None, stream=None):
    """Backward pass of jamba_ssm_gated_scan: the gradients given dout = dL/dout
    (contiguous, the dtype of x) and optionally dh_final = dL/dh_final [batch,
    d_inner] fp32.

    Returns a dict: dx, dg, dz (None without z) like x, contiguous; drate, dbias
    [d_inner] fp32 (None where the forward had none); dh0 [batch, d_inner] fp32.
    Rows of a packed batch that belong to no sequence are not written.  ``ckpt``:
    what the forward stored; without it the backward runs the recurrence once
    more.  ``workspace``: scratch of jamba_ssm_gated_scan_bwd_workspace_size()
    bytes (allocated here when None)."""
    dev = cuda_device(x, "x", "jamba_ssm_gated_scan_bwd")
    batch, seqlen, rows, d = _sizes(x, cu_seqlens, dev)
    io, shape = x.dtype, x.shape
    xs = row_stride(x, "x", shape, io, dev)
    gs = row_stride(g, "g", shape, io, dev, required=True)
    zs = row_stride(z, "z", shape, io, dev)
    need(dout, "dout", shape, io, dev)
    check(rate, "rate", (d,), _F32, dev)
    check(bias, "bias", (d,), _F32, dev)
    check(h0, "h0", (batch, d), _F32, dev)
    check(dh_final, "dh_final", (batch, d), _F32, dev)
    if ckpt is not None:
        check(ckpt, "ckpt", (rows // _lib.GATED_CKPT_STEPS + batch, d), _F32, dev)
    L = _lib.gated_lib()
    with launching(stream, dev):
        if workspace is None:
            size = L.jamba_ssm_gated_scan_bwd_workspace_size(batch, rows, d, ckpt is not None)
            workspace = x.new_empty(size, dtype=torch.uint8)
        ws, ws_bytes = _workspace(workspace, dev)
        dx, dg = empty_like(dout), empty_like(dout)
        dz = None if z is None else empty_like(dout)
        drate = None if rate is None else empty_like(rate)
        dbias = None if bias is None else empty_like(bias)
        dh0 = x.new_empty((batch, d), dtype=_F32)
        p = _lib.GatedScanBwdParams(_BWD, batch, seqlen, d, IO[io], 0, x.data_ptr(), g.data_ptr(),
                                    ptr(z), xs, gs, zs, ptr(rate), ptr(bias), ptr(h0), ptr(dout),
                                    ptr(dh_final), ptr(dx), ptr(dg), ptr(dz), ptr(drate),
                                    ptr(dbias), ptr(dh0), ptr(cu_seqlens), rows, ptr(ckpt), ws,
                                    ws_bytes)
        st = L.jamba_ssm_gated_scan_bwd(byref(p), raw_stream(dev))
    if st != _lib.OK:
        _raise(st, "jamba_ssm_gated_scan_bwd")
    return {"dx": dx, "dg": dg, "dz": dz, "drate": drate, "dbias": dbias, "dh0": dh0}


def jamba_ssm_gated_state_update(state, x, g, z=None, rate=None, bias=None, out=None,
                                 state_indices=None, workspace=None, stream=None):
    """One token for each request; `state` [batch, d_inner] fp32 is updated in
    place.  x, g, z [batch, d_inner] (rows may be strided).  With
    ``state_indices`` (int32 [batch]) `state` is a [num_slots, d_inner] cache and
    request b updates row state_indices[b], as it is: a new request's row holds
    zeros, or it takes its first token through jamba_ssm_gated_scan with
    initial_indices; a negative index skips the request (its out row is left as
    it was).  Returns out [batch, d_inner]."""
    dev = cuda_device(x, "x", "jamba_ssm_gated_state_update")
    if x.dtype not in IO:
        raise TypeError(f"x must be bfloat16 or float32, got {x.dtype}")
    if x.dim() != 2:
        raise ValueError(f"x must be [batch, d_inner], got {tuple(x.shape)}")
    io, shape = x.dtype, x.shape
    batch, d = shape
    xs = row_stride(x, "x", shape, io, dev)
    gs = row_stride(g, "g", shape, io, dev, required=True)
    zs = row_stride(z, "z", shape, io, dev)
    check(rate, "rate", (d,), _F32, dev)
    check(bias, "bias", (d,), _F32, dev)
    slots = 0
    if state_indices is not None:
        check(state_indices, "state_indices", (batch,), _I32, dev)
        slots = state.shape[0] if isinstance(state, torch.Tensor) else 0
    need(state, "state", (batch if state_indices is None else slots, d), _F32, dev)
    check(out, "out", shape, io, dev)
    ws, ws_bytes = _workspace(workspace, dev)
    with launching(stream, dev):
        if out is None:
            out = empty_like(x, xs == 0)
        p = _lib.GatedStateUpdateParams(_UPDATE, batch, d, IO[io], 0, state.data_ptr(),
                                        x.data_ptr(), g.data_ptr(), ptr(z), xs, gs, zs, ptr(rate),
                                        ptr(bias), ptr(out), ptr(state_indices), slots, ws,
                                        ws_bytes)
        st = _lib.gated_lib().jamba_ssm_gated_state_update(byref(p), raw_stream(dev))
    if st != _lib.OK:
        _raise(st, "jamba_ssm_gated_state_update")
    return out


def jamba_ssm_gated_get_status(stream=None, device=None, workspace=None) -> int:
    """Wait for the stream, then read and clear a status word: the workspace's,
    or the device's word of this library when none is given."""
    dev = status_device(stream, device, workspace)
    ws, _ = _workspace(workspace, dev)
    with launching(stream, dev):
        return _lib.gated_lib().jamba_ssm_gated_get_status(ws, raw_stream(dev))
