"""Marshalling of strided [B, heads, n, d] tensors and of streams for the calls that take views.

A call's arguments go to the library as one packed structure of include/anchor_attn.h: the smallest calls take a few
microseconds on the device, and building ctypes structures field by field took longer than that."""
from __future__ import annotations

import torch

DTYPES = {torch.bfloat16: 0, torch.float32: 1}
VIEW = "Qqqq"              # anchor_attn_view_t: pointer, batch, head and row strides
NO_VIEW = (0, 0, 0, 0)

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


_package = None


def library():
    """The package's loaded library."""
    global _package
    if _package is None:
        import linear_complexity_anchor_gb300
        _package = linear_complexity_anchor_gb300
    return _package._lib or _package.load()


def fail(status: int, what: str) -> None:
    _package._raise(status, what)


def rows_dtype(t, name: str) -> int:
    """The ABI's number of a CUDA tensor's type."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dt = DTYPES.get(t.dtype)
    if dt is None:
        raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    if t.get_device() < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dt


def view(t, name: str, dtype, device: int) -> tuple:
    """(pointer, strides) of a four-axis tensor of this type, on this CUDA device, whose last axis is dense."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device}, got {t.device}")
    strides = t.stride()
    if len(strides) != 4:
        raise ValueError(f"{name} must have 4 axes, got {len(strides)}")
    if strides[3] != 1 and t.size(3) > 1:
        raise ValueError(f"the last axis of {name} must be dense")
    return t.data_ptr(), strides[0], strides[1], strides[2]


def empty_like(t):
    """A tensor of t's shape, with t's order of axes where t is dense, and its view."""
    r = torch.empty_like(t)
    strides = r.stride()
    if strides[3] != 1 and r.size(3) > 1:
        r = torch.empty(t.shape, dtype=t.dtype, device=t.device)
        strides = r.stride()
    return r, (r.data_ptr(), strides[0], strides[1], strides[2])


class Launch:
    """The device and stream of one call: `with Launch(device, stream) as handle`.  Tensors made inside belong to that
    stream; where `stream` is not None, `used(...)` tells the allocator of tensors that are used on a
    stream other than their own."""

    __slots__ = ("device", "handle", "stream", "current", "guards")

    def __init__(self, device: int, stream=None):
        self.device, self.stream, self.guards = device, None, ()
        if stream is None and _raw_stream is not None:
            self.handle = _raw_stream(device)
            return
        self.current = torch.cuda.current_stream(device)
        stream = self.current if stream is None else stream
        if stream.device.index != device:
            raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{device}")
        self.handle = stream.cuda_stream
        if stream != self.current:
            self.stream = stream

    def __enter__(self) -> int:
        if self.stream is not None:
            self.guards = (torch.cuda.device(self.device), torch.cuda.stream(self.stream))
        elif _current_device() != self.device:
            self.guards = (torch.cuda.device(self.device),)
        for g in self.guards:
            g.__enter__()
        return self.handle

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)

    def used(self, given, made=()) -> None:
        """For a call whose `stream` is not None: the caller's tensors, outputs among them, are used on it; those made
        inside are the stream's own, and the caller uses them on its current one."""
        for t in given:
            if t is not None:
                t.record_stream(self.stream)
        for t in made:
            if t is not None:
                t.record_stream(self.current)
