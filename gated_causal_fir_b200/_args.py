"""Checks of arguments, launch contexts and workspaces shared by the mixer operators' bindings.

A call for one token takes a few microseconds on the device, so the checks are written to cost
little where they pass; what is wrong is found out only once something is.
"""
import functools

from . import _native
from ._native import HYENA_DTYPE_BF16, HYENA_DTYPE_F32

_TORCH = None
_CODES = {}


def torch_():
    global _TORCH
    if _TORCH is None:
        import torch
        _CODES.update({torch.bfloat16: HYENA_DTYPE_BF16, torch.float32: HYENA_DTYPE_F32})
        _TORCH = torch
    return _TORCH


def code(t, what):
    """The HYENA_DTYPE_* of a tensor."""
    torch_()
    c = _CODES.get(t.dtype)
    if c is None:
        raise TypeError("%s must be bfloat16 or float32, got %s" % (what, t.dtype))
    return c


def cuda_tensor(name, t, what):
    if not isinstance(t, torch_().Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA %s" % (name, what))


def need(name, t, shape, dtype, device):
    """``t`` must be a contiguous tensor of this shape and type on this (CUDA) device."""
    try:
        if t.shape == shape and t.dtype is dtype and t.device == device and t.is_contiguous():
            return t
    except AttributeError:
        pass
    cuda_tensor(name, t, "tensor")
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.device != device:
        raise ValueError("%s is on %s, the first input on %s" % (name, t.device, device))
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    raise ValueError("%s must be contiguous" % name)


def ptr(t):
    return None if t is None else t.data_ptr()


class On:
    """The launch context of a call: the tensors' device made current, and the stream (by default
    that device's current one).  ``keep`` marks buffers made here as in use on a given stream."""
    __slots__ = ("given", "handle", "guard")

    def __init__(self, device, stream):
        torch = torch_()
        self.given = stream
        self.handle = (torch._C._cuda_getCurrentRawStream(device.index) if stream is None
                       else stream.cuda_stream)
        self.guard = (None if device.index == torch._C._cuda_getDevice()
                      else torch.cuda.device(device))

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)

    def keep(self, *tensors):
        if self.given is not None:
            for t in tensors:
                t.record_stream(self.given)


def workspace(given, size, device, on):
    """(pointer, bytes) of the workspace: the caller's, or one made here; (None, 0) for none."""
    if given is None:
        if size == 0:
            return None, 0
        ws = torch_().empty(size, dtype=torch_().uint8, device=device)
        on.keep(ws)
        return ws.data_ptr(), size
    if not isinstance(given, torch_().Tensor) or given.device != device \
            or not given.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on the inputs' device")
    return given.data_ptr(), given.numel() * given.element_size()


@functools.lru_cache(maxsize=4096)
def nbytes(fn, *args):
    """A host-only size query of the library (the same answer for the same sizes)."""
    n = int(getattr(_native.lib(), fn)(*args))
    if n < 0:
        raise _native.HyenaError(fn, -n)
    return n
