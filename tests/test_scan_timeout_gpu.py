"""Failure detection of the recurrence's clusters, made to fire without faulting the GPU (needs a
B200).

The CTAs of a cluster wait for each other's (A, S) within a bound.  hyena_testing_scan_fault
shortens it to 20 ms and withholds one: every CTA must leave, HYENA_DEVICE_TIMEOUT be raised, and
the next ordinary call be right."""
import time

import pytest
import torch

import gated_causal_fir_b200 as g
from gated_causal_fir_b200 import _native
from tests import _scan_ref as R
from tests.test_scan_gpu import make

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
WAIT_NS = 20 * 1000 * 1000
SHAPES = [(1, 1250, 320, 64), (2, 1500, 128, 4), (1, 2500, 36, 1)]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from gated_causal_fir_b200 import build
    build.build()
    g.hyena_device_status(clear=True)
    yield
    assert g.hyena_device_status(clear=True) == 0, "a kernel raised its device status word"


def call(q, k, v, lg, y, s_out, d_g, fault):
    return _native.lib().hyena_testing_scan_fault(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), lg.data_ptr(), y.data_ptr(), s_out.data_ptr(),
        *q.shape, d_g, 1 if q.dtype == F32 else 0, fault, WAIT_NS,
        torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "f32"))
@pytest.mark.parametrize("shape", SHAPES, ids=["x".join(map(str, s)) for s in SHAPES])
def test_a_cluster_that_waits_in_vain_gives_up(shape, dtype):
    B, L, D, d_g = shape
    q, k, v, lg, _, _, _ = make(B, L, D, d_g, dtype)
    y, s_out = torch.empty_like(q), torch.empty(B, D, device="cuda")
    ref = R.Ref(q, k, v, lg, d_g, None)
    assert call(q, k, v, lg, y, s_out, d_g, 0) == _native.HYENA_OK
    R.check("y", y, ref)
    assert g.hyena_device_status(clear=True) == 0
    t0 = time.perf_counter()
    assert call(q, k, v, lg, y, s_out, d_g, 1) == _native.HYENA_OK
    torch.cuda.synchronize()
    took = time.perf_counter() - t0
    assert g.hyena_device_status(clear=True) & g.HYENA_DEVICE_TIMEOUT
    assert took < 1.0, "the timed-out kernel took %.3f s" % took
    y, s_out = g.hyena_scan_fwd(q, k, v, lg, d_g)
    R.check("y", y, ref)
    R.check("s_out", s_out, ref)
    assert g.hyena_device_status(clear=True) == 0
