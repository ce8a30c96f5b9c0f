"""Marshalling of strided [B, heads, n, d] tensors and of streams for the calls that take views."""
from __future__ import annotations

import contextlib
import ctypes

DTYPES = {"torch.bfloat16": 0, "torch.float32": 1}


class View(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("batch", ctypes.c_longlong), ("head", ctypes.c_longlong),
                ("row", ctypes.c_longlong)]


NO_VIEW = View()


def view(t) -> View:
    sb, sh, sn, _ = t.stride()
    return View(t.data_ptr(), sb, sh, sn)


def rows_dtype(t, name: str) -> int:
    dt = DTYPES.get(str(t.dtype))
    if dt is None:
        raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    return dt


def check(t, name: str, like=None, dim: int = 4) -> None:
    """A CUDA tensor of `like`'s type and device, whose last axis is dense."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if like is not None:
        if t.dtype != like.dtype:
            raise TypeError(f"{name} must be {like.dtype}, got {t.dtype}")
        if t.device != like.device:
            raise ValueError(f"{name} must be on {like.device}, got {t.device}")
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} axes, got {t.dim()}")
    if t.size(-1) > 1 and t.stride(-1) != 1:
        raise ValueError(f"the last axis of {name} must be dense")


def empty_like(t):
    """A tensor of t's shape, with t's order of axes where t is dense."""
    import torch
    r = torch.empty_like(t)
    return r if r.size(-1) <= 1 or r.stride(-1) == 1 else torch.empty(t.shape, dtype=t.dtype, device=t.device)


@contextlib.contextmanager
def _both(device, stream):
    import torch
    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield


class Launch:
    """The device and stream of one call: `with Launch(device, stream) as handle`.  Tensors made
    inside belong to that stream; `used(...)` tells the allocator of tensors that are used on a
    stream other than their own."""

    __slots__ = ("device", "stream", "current", "guard")

    def __init__(self, device, stream=None):
        import torch
        self.device = device
        self.current = torch.cuda.current_stream(device)
        self.stream = self.current if stream is None else stream
        if self.stream.device != device:
            raise ValueError(f"stream is on {self.stream.device}, the tensors on {device}")
        self.guard = None

    def __enter__(self) -> int:
        import torch
        if self.stream != self.current:
            self.guard = _both(self.device, self.stream)
        elif torch.cuda.current_device() != self.device.index:
            self.guard = torch.cuda.device(self.device)
        if self.guard is not None:
            self.guard.__enter__()
        return self.stream.cuda_stream

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)
            self.guard = None

    def used(self, inputs, outputs=()) -> None:
        if self.stream != self.current:
            for t in inputs:
                if t is not None:
                    t.record_stream(self.stream)
            for t in outputs:
                if t is not None:
                    t.record_stream(self.current)
