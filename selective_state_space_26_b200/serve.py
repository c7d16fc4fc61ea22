"""What a serving step needs around the scans: binding of
include/jamba_ssm_serve.h.

* ``jamba_ssm_i8_quant`` / ``jamba_ssm_i8_proj`` -- the layer's large
  projections in 8-bit integers, a scale for each token and output channel;
* ``jamba_ssm_batch_maps`` -- cu_seqlens, positions, block tables, cache slots
  and state slots of a continuous batch, from its requests' lengths.

Every step runs in the kernels of libjamba_ssm_serve.so; this module checks
tensor metadata, allocates outputs and hands over pointers and the stream.
"""
from __future__ import annotations

from ctypes import byref, sizeof

import torch

from . import _lib
from ._lib import JambaSSMError
from ._tensors import (IO, check, cuda_device, launching, need, ptr, raw_stream, row_stride,
                       status_device)

__all__ = ["jamba_ssm_i8_quant", "jamba_ssm_i8_proj", "jamba_ssm_batch_maps",
           "jamba_ssm_serve_get_status"]

_F32, _I8, _I32, _I64 = torch.float32, torch.int8, torch.int32, torch.int64
_QUANT, _PROJ, _MAPS = (sizeof(c) for c in (_lib.I8QuantParams, _lib.I8ProjParams,
                                            _lib.BatchMapsParams))


def _raise(status, what):
    raise JambaSSMError(status, what, cuda_error=_lib.serve_lib().jamba_ssm_serve_last_cuda_error())


def jamba_ssm_i8_quant(x, q=None, scale=None, stream=None):
    """Rows to 8 bits: scale = max|x| / 127 over each row, q = x / scale rounded
    to the nearest integer.  x [..., k] bf16 or fp32 (rows may be evenly
    strided).  Returns (q, scale): q int8 [..., k rounded up to 16], the columns
    behind k zero, and scale fp32 [...].  The same call lays out a weight
    [n_out, k] once, one scale for each output channel."""
    dev = cuda_device(x, "x", "jamba_ssm_i8_quant")
    if x.dtype not in IO:
        raise TypeError(f"x must be bfloat16 or float32, got {x.dtype}")
    if x.dim() < 1:
        raise ValueError("x must be [..., k]")
    k, lead = x.shape[-1], x.shape[:-1]
    xs = row_stride(x, "x", x.shape, x.dtype, dev)
    pitch = (k + 15) // 16 * 16
    rows = lead.numel()
    check(q, "q", (*lead, pitch), _I8, dev)
    check(scale, "scale", lead, _F32, dev)
    with launching(stream, dev):
        if q is None:
            q = x.new_empty((*lead, pitch), dtype=_I8)
        if scale is None:
            scale = x.new_empty(lead, dtype=_F32)
        p = _lib.I8QuantParams(_QUANT, rows, k, IO[x.dtype], 0, x.data_ptr(), xs, q.data_ptr(),
                               scale.data_ptr())
        st = _lib.serve_lib().jamba_ssm_i8_quant(byref(p), raw_stream(dev))
    if st != _lib.OK:
        _raise(st, "jamba_ssm_i8_quant")
    return q, scale


def jamba_ssm_i8_proj(q, q_scale, w, w_scale, bias=None, out=None, out_dtype=torch.bfloat16,
                      timeout_cycles: int = 0, stream=None, debug_flags: int = 0):
    """out = (q . w) * q_scale * w_scale + bias, the sum exact in 32-bit
    integers, rounded once to out_dtype (bf16 or fp32).  A token's outputs have
    the same bits whatever batch it is in.

    q int8 [..., pitch] and q_scale fp32 [...] of jamba_ssm_i8_quant; w int8
    [n_out, pitch] and w_scale fp32 [n_out] of the same call on the weight; bias
    fp32 [n_out] or None.  Returns out [..., n_out]."""
    dev = cuda_device(q, "q", "jamba_ssm_i8_proj")
    if q.dim() < 1 or q.shape[-1] % 16:
        raise ValueError(f"q must be [..., a multiple of 16], got {tuple(q.shape)}")
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w must be a tensor [n_out, pitch]")
    if out is not None:
        out_dtype = out.dtype
    if out_dtype not in IO:
        raise TypeError(f"out_dtype must be bfloat16 or float32, got {out_dtype}")
    pitch, lead, n = q.shape[-1], q.shape[:-1], w.shape[0]
    check(q, "q", q.shape, _I8, dev)
    need(q_scale, "q_scale", lead, _F32, dev)
    need(w, "w", (n, pitch), _I8, dev)
    need(w_scale, "w_scale", (n,), _F32, dev)
    check(bias, "bias", (n,), _F32, dev)
    check(out, "out", (*lead, n), out_dtype, dev)
    with launching(stream, dev):
        if out is None:
            out = q.new_empty((*lead, n), dtype=out_dtype)
        p = _lib.I8ProjParams(_PROJ, lead.numel(), pitch, n, IO[out_dtype], 0,
                              q.data_ptr(), q_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(),
                              ptr(bias), out.data_ptr(), int(timeout_cycles), int(debug_flags))
        st = _lib.serve_lib().jamba_ssm_i8_proj(byref(p), raw_stream(dev))
    if st != _lib.OK:
        _raise(st, "jamba_ssm_i8_proj")
    return out


def jamba_ssm_batch_maps(new_lens, block_tables, free_blocks, request_slots, free_slots,
                         ctx_lens=None, block_size=16, max_tokens=None, stream=None):
    """The maps of one step of a continuous batch, in one launch.

    new_lens, ctx_lens (None: zeros) int32 [requests]: the tokens each request
    brings, and those it had before.  block_tables int32 [requests, max_blocks]
    and request_slots int32 [requests] are updated in place: a request takes the
    cache blocks it needs beyond those of its context from free_blocks, and a
    request without context takes a state slot from free_slots, both in order.
    max_tokens: rows of the per-token maps, at least the batch's tokens (the
    host's bound; rows behind the batch hold -1).

    Returns a dict: cu_seqlens [requests + 1], positions, token_request
    [max_tokens], slot_map int64 [max_tokens], block_tables, request_slots,
    state_indices, initial_indices [requests], counts [4] = tokens, blocks
    taken, slots taken, longest request.  initial_indices lets the gated scan
    start a new request from zero; jamba_ssm_scan and the one-token updates read
    the row of its slot: for them zero the row (``cache[slot] = 0``) when the
    request that held it ends, before the slot is in free_slots again.  What does not fit (tokens past
    max_tokens, no free block or slot, a request longer than its table) is
    recorded in the status word (jamba_ssm_serve_get_status)."""
    dev = cuda_device(new_lens, "new_lens", "jamba_ssm_batch_maps")
    for t, name in ((block_tables, "block_tables"), (free_blocks, "free_blocks"),
                    (free_slots, "free_slots")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    if new_lens.dim() != 1 or block_tables.dim() != 2:
        raise ValueError("new_lens must be [requests] and block_tables [requests, max_blocks]")
    if max_tokens is None:
        raise ValueError("max_tokens is needed: the rows of the per-token maps")
    if max_tokens < 0 or block_size < 1:
        raise ValueError("max_tokens must be >= 0 and block_size >= 1")
    n, width = new_lens.shape[0], block_tables.shape[1]
    check(new_lens, "new_lens", (n,), _I32, dev)
    check(ctx_lens, "ctx_lens", (n,), _I32, dev)
    need(block_tables, "block_tables", (n, width), _I32, dev)
    need(request_slots, "request_slots", (n,), _I32, dev)
    check(free_blocks, "free_blocks", free_blocks.shape, _I32, dev)
    check(free_slots, "free_slots", free_slots.shape, _I32, dev)
    t = int(max_tokens)
    with launching(stream, dev):
        # one buffer, the per-token maps first, each of them from a multiple of 16 bytes on
        r = -t % 4
        buf = new_lens.new_empty(4 * (t + r) + 3 * n + 5)
        if r:
            slot_map, _, pos, _, req, _, cu, si, ii, counts = buf.split_with_sizes(
                (2 * t, 2 * r, t, r, t, r, n + 1, n, n, 4))
        else:
            slot_map, pos, req, cu, si, ii, counts = buf.split_with_sizes(
                (2 * t, t, t, n + 1, n, n, 4))
        slot_map = slot_map.view(_I64)
        base = buf.data_ptr()
        at_pos = base + 8 * (t + r)
        at_req = at_pos + 4 * (t + r)
        at_cu = at_req + 4 * (t + r)
        at_si = at_cu + 4 * (n + 1)
        p = _lib.BatchMapsParams(
            _MAPS, n, t, width, int(block_size), new_lens.data_ptr(), ptr(ctx_lens),
            free_blocks.data_ptr(), free_blocks.numel(), free_slots.data_ptr(),
            free_slots.numel(), block_tables.data_ptr(), request_slots.data_ptr(), at_cu, at_pos,
            at_req, base, at_si, at_si + 4 * n, at_si + 8 * n)
        st = _lib.serve_lib().jamba_ssm_batch_maps(byref(p), raw_stream(dev))
    if st != _lib.OK:
        _raise(st, "jamba_ssm_batch_maps")
    return {"cu_seqlens": cu, "positions": pos, "token_request": req, "slot_map": slot_map,
            "block_tables": block_tables, "request_slots": request_slots, "state_indices": si,
            "initial_indices": ii, "counts": counts}


def jamba_ssm_serve_get_status(stream=None, device=None) -> int:
    """Wait for the stream, then read and clear this library's status word."""
    dev = status_device(stream, device)
    with launching(stream, dev):
        return _lib.serve_lib().jamba_ssm_serve_get_status(raw_stream(dev))
