"""Checks of arguments, launch contexts and workspaces shared by the mixer operators' bindings.

A call for one token takes a few microseconds on the device, so the checks are written to cost
little where they pass; what is wrong is found out only once something is.
"""
import functools

from . import _native
from ._native import HYENA_DTYPE_BF16, HYENA_DTYPE_F32

_TORCH = None
CODES = {}
_FUNCTIONS = {}


def torch_():
    global _TORCH
    if _TORCH is None:
        import torch
        CODES.update({torch.bfloat16: HYENA_DTYPE_BF16, torch.float32: HYENA_DTYPE_F32})
        _TORCH = torch
    return _TORCH


def code(t, what):
    """The HYENA_DTYPE_* of a tensor."""
    torch_()
    c = CODES.get(t.dtype)
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


def like(t, shape, dtype, device):
    """Whether ``t`` is what need() asks for."""
    return (t.dtype is dtype and t.shape == shape and t.device == device
            and t.is_contiguous())


def ptr(t):
    return None if t is None else t.data_ptr()


def stream_handle(device, stream):
    """The raw handle of ``stream``, by default the current one of ``device``."""
    return (torch_()._C._cuda_getCurrentRawStream(device.index) if stream is None
            else stream.cuda_stream)


def made(stream, device, make):
    """make(), a buffer for a call on the stream that the caller gave (None: the current one).

    The buffer comes from that stream's memory: one from the current stream's could have been in use
    a moment ago by work that is still queued there, which the given stream does not wait for.  The
    current stream is told of it too, since results are read and dropped there."""
    if stream is None:
        return make()
    torch = torch_()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=device)
    current = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        t = make()
    if stream != current:
        t.record_stream(current)
    return t


def run(name, device, *args):
    """Calls a function of the library with the tensors' device current; raises on an error."""
    torch = torch_()
    fn = _FUNCTIONS.get(name)
    if fn is None:
        fn = _FUNCTIONS[name] = getattr(_native.lib(), name)
    if device.index == torch._C._cuda_getDevice():
        rc = fn(*args)
    else:
        with torch.cuda.device(device):
            rc = fn(*args)
    if rc:
        _native.check(name, rc)


def workspace(given, size, device, stream):
    """(pointer, bytes, buffer) of the workspace: the caller's, or one made here; none for 0."""
    if given is None:
        if size == 0:
            return None, 0, None
        ws = made(stream, device,
                  lambda: torch_().empty(size, dtype=torch_().uint8, device=device))
        return ws.data_ptr(), size, ws
    if not isinstance(given, torch_().Tensor) or given.device != device \
            or not given.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on the inputs' device")
    return given.data_ptr(), given.numel() * given.element_size(), given


@functools.lru_cache(maxsize=4096)
def nbytes(fn, *args):
    """A host-only size query of the library (the same answer for the same sizes)."""
    n = int(getattr(_native.lib(), fn)(*args))
    if n < 0:
        raise _native.HyenaError(fn, -n)
    return n
