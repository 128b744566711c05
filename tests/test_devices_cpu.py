"""Calls for tensors on a device that is not the current one, on the CPU: fakes stand for the CUDA
tensors and for the library, and show which device is current, and which stream is given, when the
library is called."""
import contextlib

import pytest
import torch

import gated_causal_fir_b200 as g
from gated_causal_fir_b200 import _args, _native


class Fake(torch.Tensor):
    """A host tensor that says it is on cuda:1."""
    is_cuda = True
    index = 1

    @property
    def device(self):
        return torch.device("cuda", self.index)


class Other(Fake):
    index = 0


def fake(*shape, dtype=torch.bfloat16, cls=Fake):
    return torch.zeros(*shape, dtype=dtype).as_subclass(cls)


@pytest.fixture
def calls(monkeypatch):
    """The library's calls as (name, current device, last argument)."""
    log, current = [], [0]

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], torch.device(d).index
        yield
        current[0] = before

    class Library:
        def __getattr__(self, name):
            def fn(*args):
                log.append((name, current[0], getattr(args[-1], "value", args[-1])))
                return 0
            return fn

    _args.torch_()
    monkeypatch.setattr(_args, "_FUNCTIONS", {})
    monkeypatch.setattr(_native, "lib", Library)
    monkeypatch.setattr(_args, "nbytes", lambda *a: 0)
    for module in ("projection", "recurrence"):
        monkeypatch.setattr("gated_causal_fir_b200.%s.nbytes" % module, lambda *a: 0)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 1000 + i, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: type(
        "S", (), {"cuda_stream": 1000 + (current[0] if d is None else torch.device(d).index)})())
    return log


def small():
    q, k, v, dy = (fake(1, 8, 16) for _ in range(4))
    return q, k, v, dy, fake(2, 4, dtype=torch.float32)


CALLS = {
    "hyena_conv_fwd": lambda q, k, v, dy, h: g.hyena_conv_fwd(q, k, v, h, 8, 4),
    "hyena_conv_fwd_ex": lambda q, k, v, dy, h: g.hyena_conv_fwd_ex(q, k, v, h, 8, 4),
    "hyena_conv_fwd_f32": lambda q, k, v, dy, h: g.hyena_conv_fwd_f32(
        *(t.float() for t in (q, k, v)), h, 8, 4),
    "hyena_conv_fwd_hist": lambda q, k, v, dy, h: g.hyena_conv_fwd_hist(q, k, v, h, 8, 4, k, v),
    "hyena_conv_fwd_fft": lambda q, k, v, dy, h: g.hyena_conv_fwd_fft(
        q, k, v, h, 8, 4, workspace=fake(256, dtype=torch.uint8)),
    "hyena_conv_bwd_ex": lambda q, k, v, dy, h: g.hyena_conv_bwd(
        q, k, v, h, dy, 8, 4, workspace=fake(256, dtype=torch.uint8)),
    "hyena_scan_fwd": lambda q, k, v, dy, h: g.hyena_scan_fwd(
        q, k, v, dy, 1, s0=fake(1, 16, dtype=torch.float32)),
    "hyena_proj_fwd": lambda q, k, v, dy, h: g.hyena_proj_fwd(q, fake(24, 16)),
    "mixer with the FIR": lambda q, k, v, dy, h: g.hyena_mixer_fwd(
        q, g.MixerParams(*(g.Linear(fake(16, 16)) for _ in range(4)), 8, filters=h)),
}


@pytest.mark.parametrize("name", CALLS)
def test_the_tensors_device_is_current_and_its_stream_is_used(name, calls):
    CALLS[name](*small())
    launches = [c for c in calls if "bytes" not in c[0]]
    assert launches and all(c[1:] == (1, 1001) for c in launches), launches
    if name.startswith("hyena"):
        assert launches[-1][0] == name
    assert torch._C._cuda_getDevice() == 0


@pytest.mark.parametrize("which", range(5))
def test_tensors_on_two_devices_are_refused(which, calls):
    args = list(small())
    args[which] = args[which].as_subclass(Other)
    q, k, v, dy, h = args
    with pytest.raises(ValueError):
        if which == 3:
            g.hyena_conv_bwd(q, k, v, h, dy, 8, 4, workspace=fake(256, dtype=torch.uint8))
        else:
            g.hyena_conv_fwd(q, k, v, h, 8, 4)
    with pytest.raises(ValueError):
        g.hyena_conv_fwd(*(small()[i] for i in (0, 1, 2, 4)), 8, 4,
                         y=fake(1, 8, 16, cls=Other))
    assert not [c for c in calls if "bytes" not in c[0]]
