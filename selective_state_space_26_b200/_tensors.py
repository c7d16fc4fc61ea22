"""Checks of tensor arguments and the choice of device and stream, shared by the
gated recurrence's and the serving step's bindings."""
from __future__ import annotations

import contextlib

import torch

from . import _lib

IO = {torch.bfloat16: _lib.BF16, torch.float32: _lib.F32}
_HERE = contextlib.nullcontext()


def ptr(t):
    return None if t is None else t.data_ptr()


def check(t, name, shape, dtype, device):
    """A contiguous tensor of this shape, dtype and device (or None)."""
    if t is None:
        return
    try:  # the usual case first: these calls are made per token
        if (t.dtype is dtype and t.shape == shape and t.device == device
                and t.is_contiguous()):
            return
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def need(t, name, shape, dtype, device):
    """As check, for a tensor that must be there."""
    if t is None:
        raise TypeError(f"{name} must be a torch.Tensor")
    check(t, name, shape, dtype, device)


def row_stride(t, name, shape, dtype, device, required=False):
    """Elements between the rows of an activation whose channels are contiguous
    and whose rows are evenly spaced (0 for None or a contiguous tensor)."""
    if t is None and not required:
        return 0
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is dtype and t.shape == shape and t.device == device:  # the usual cases first
        if t.is_contiguous():
            return 0
        if t.dim() == 2 and t.stride(1) == 1 and t.stride(0) >= shape[1] and shape[0] > 1:
            return t.stride(0)
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.is_contiguous():
        return 0
    # the dimensions before the channels, outermost first, those of one row left out
    dims = [(n, s) for n, s in zip(t.shape[:-1], t.stride()[:-1]) if n != 1]
    width = t.shape[-1]
    even = all(dims[i][1] == dims[i + 1][0] * dims[i + 1][1] for i in range(len(dims) - 1))
    if (width > 1 and t.stride(-1) != 1) or not even or (dims and dims[-1][1] < width):
        raise ValueError(f"{name} must have contiguous channels and evenly spaced rows "
                         f"(shape {tuple(t.shape)}, strides {t.stride()})")
    return dims[-1][1] if dims else 0


def cuda_device(t, name, what):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{what} needs CUDA tensors; there is no CPU path")
    return t.device


def _device_of(stream):
    """The device of a stream that says it (None: a raw handle)."""
    dev = getattr(stream, "device", None)
    return dev if isinstance(dev, torch.device) else None


def launching(stream, device):
    """Context for a call's allocations and launch: the tensors' device is the
    current one and, where the caller names a stream, that stream too, so what
    is allocated for the call belongs to the stream that uses it."""
    if stream is None:
        return _HERE if torch.cuda.current_device() == device.index else torch.cuda.device(device)
    # the kernel would run on the stream's device, with the tensors' addresses
    if _device_of(stream) not in (None, device):
        raise ValueError(f"stream is on {stream.device}, expected {device}")
    if not isinstance(stream, torch.cuda.Stream):
        raw = int(getattr(stream, "cuda_stream", stream))
        stream = torch.cuda.ExternalStream(raw, device=device) if raw else \
            torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def status_device(stream, device, workspace=None):
    """The device, with its index, of a status word: of the named one, the
    workspace or the stream, the first that is given, else the current one."""
    dev = device if device is not None else workspace.device if workspace is not None else \
        _device_of(stream)
    dev = torch.device("cuda" if dev is None else dev)
    return dev if dev.index is not None else torch.device(dev.type, torch.cuda.current_device())


def raw_stream(device):
    """The device's current stream, without making a Stream object for it."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def empty_like(t, contiguous=True):
    """An uninitialised contiguous tensor like t (`contiguous`: whether t is)."""
    if contiguous:
        return torch.empty_like(t)
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def workspace(ws, device):
    """(pointer, bytes) of an optional workspace tensor."""
    if ws is None:
        return None, 0
    if not isinstance(ws, torch.Tensor) or ws.device != device or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the device of the inputs")
    return ws.data_ptr(), ws.numel() * ws.element_size()
