"""Failure detection of the projections, made to fire without faulting the GPU (needs a B200).

The waits between the kernel's warps are bounded.  hyena_testing_proj_fault shortens the bound to
20 ms and withholds what one of them waits for: the kernel must raise HYENA_DEVICE_TIMEOUT, let
every role leave, wait for its copies and MMAs in flight, free tensor memory and return well within
a second, and the next ordinary call must be right."""
import time

import pytest
import torch

import gated_causal_fir_b200 as g
from gated_causal_fir_b200 import _native

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
WAIT_NS = 20 * 1000 * 1000
# tiles of one CTA, and (the last) of pairs of CTAs
SHAPES = [(300, 256, 64), (300, 256, 200), (9472, 512, 2048)]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from gated_causal_fir_b200 import build
    build.build()
    g.hyena_device_status(clear=True)
    yield
    assert g.hyena_device_status(clear=True) == 0, "a kernel raised its device status word"


def make(M, N, K):
    gen = torch.Generator(device="cuda").manual_seed(M + N)
    r = lambda *s: torch.randint(-2, 3, s, generator=gen, device="cuda").to(BF16)  # noqa: E731
    x, w, res = r(M, K), r(N, K), r(M, N)
    # sums of small integers: exact before the one rounding
    return x, w, res, (x.double() @ w.double().t() + res.double()).to(BF16)


def call(x, w, res, y, fault):
    M, K = x.shape
    rc = _native.lib().hyena_testing_proj_fault(
        x.data_ptr(), w.data_ptr(), res.data_ptr(), y.data_ptr(), M, w.shape[0], K, fault, WAIT_NS,
        torch.cuda.current_stream().cuda_stream)
    assert rc == _native.HYENA_OK


@pytest.mark.parametrize("shape", SHAPES, ids=["x".join(map(str, s)) for s in SHAPES])
def test_short_limit_without_fault_runs_normally(shape):
    x, w, res, want = make(*shape)
    y = torch.empty_like(res)
    call(x, w, res, y, 0)
    assert torch.equal(y, want) and g.hyena_device_status(clear=True) == 0


FAULTS = {"residual never requested": 1, "accumulator never announced": 2,
          "copies of a pair end after a stage": 3}
CASES = [(s, f) for f in FAULTS for s in SHAPES if FAULTS[f] != 3 or s == SHAPES[-1]]


@pytest.mark.parametrize("shape,fault", CASES, ids=["%dx%dx%d %s" % (*s, f) for s, f in CASES])
def test_what_never_comes_is_given_up(shape, fault):
    fault = FAULTS[fault]
    x, w, res, want = make(*shape)
    y = torch.empty_like(res)
    g.hyena_proj_fwd(x, w, residual=res)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    call(x, w, res, y, fault)
    torch.cuda.synchronize()
    took = time.perf_counter() - t0
    assert g.hyena_device_status(clear=True) & g.HYENA_DEVICE_TIMEOUT
    assert took < 1.0, "the timed-out kernel took %.3f s" % took
    assert torch.equal(g.hyena_proj_fwd(x, w, residual=res), want)
    assert g.hyena_device_status(clear=True) == 0
