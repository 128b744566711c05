"""Checks of arguments, launch contexts and workspaces shared by the mixer operators' bindings."""
from . import _native
from ._native import HYENA_DTYPE_BF16, HYENA_DTYPE_F32


def torch_():
    import torch
    return torch


def code(t, what):
    torch = torch_()
    if t.dtype == torch.bfloat16:
        return HYENA_DTYPE_BF16
    if t.dtype == torch.float32:
        return HYENA_DTYPE_F32
    raise TypeError("%s must be bfloat16 or float32, got %s" % (what, t.dtype))


def need(name, t, shape, dtype, device):
    """``t`` must be a contiguous CUDA tensor of this shape and type on this device."""
    if not isinstance(t, torch_().Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.device != device:
        raise ValueError("%s is on %s, the first input on %s" % (name, t.device, device))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must be %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def ptr(t):
    return None if t is None else t.data_ptr()


class On:
    """The launch context of a call: the tensors' device made current, and the stream (by default
    that device's current one).  ``keep`` marks buffers made here as in use on a given stream."""

    def __init__(self, device, stream):
        cuda = torch_().cuda
        self._given = stream
        self.stream = cuda.current_stream(device) if stream is None else stream
        same = device.index == cuda.current_device()
        self._guard = None if same else cuda.device(device)

    def __enter__(self):
        if self._guard is not None:
            self._guard.__enter__()
        return self

    def __exit__(self, *exc):
        if self._guard is not None:
            self._guard.__exit__(*exc)

    def keep(self, *tensors):
        if self._given is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(self._given)


def workspace(given, need, device, on):
    """(pointer, bytes) of the workspace: the caller's, or one made here; (None, 0) for none."""
    torch = torch_()
    if given is not None:
        if not isinstance(given, torch.Tensor) or not given.is_cuda or given.device != device \
                or not given.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor on the inputs' device")
        return given.data_ptr(), given.numel() * given.element_size()
    if need == 0:
        return None, 0
    ws = torch.empty(need, dtype=torch.uint8, device=device)
    on.keep(ws)
    return ws.data_ptr(), need


def nbytes(fn, *args):
    n = int(getattr(_native.lib(), fn)(*args))
    if n < 0:
        raise _native.HyenaError(fn, -n)
    return n
