"""The FIR's calls on a stream that the caller gives, beside work on the current one (needs a B200);
what is asked of them is in test_mixer_streams_gpu."""
import pytest
import torch

import gated_causal_fir_b200 as g
from tests.test_mixer_streams_gpu import beside_queued_work

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from gated_causal_fir_b200 import build
    build.build()
    g.hyena_device_status(clear=True)
    yield
    assert g.hyena_device_status(clear=True) == 0, "a kernel raised its device status word"


@pytest.mark.parametrize("name", ("fwd", "hist", "fft", "bwd", "toeplitz"))
def test_a_given_stream_does_not_share_freed_memory_with_the_current_one(name):
    B, L, D, d_g, l_h = 1, 2048, 256, 64, 128
    q, k, v, dy = (torch.randn(B, L, D, device="cuda").to(BF16) for _ in range(4))
    h = torch.randn(D // d_g, l_h, device="cuda") / l_h ** 0.5
    full = torch.randn(D // d_g, L, device="cuda") / L ** 0.5
    n = q.numel() * 2
    call, sizes = {
        "fwd": (lambda s: g.hyena_conv_fwd(q, k, v, h, d_g, 64, stream=s), [n]),
        "hist": (lambda s: g.hyena_conv_fwd_hist(q, k, v, h, d_g, 64, k, v, stream=s), [n]),
        "fft": (lambda s: g.hyena_conv_fwd_fft(q, k, v, full, d_g, 64, stream=s),
                [n, g.hyena_conv_fwd_fft_workspace_bytes(B, L, D, d_g, L)]),
        "bwd": (lambda s: g.hyena_conv_bwd(q, k, v, h, dy, d_g, 64, stream=s),
                [n, h.numel() * 4, g.hyena_conv_bwd_workspace_bytes(B, L, D, d_g, l_h)]),
        "toeplitz": (lambda s: g.hyena_build_toeplitz_blocks(h, 64, stream=s),
                     [4 * 64 * 64 * 4 * S for S in (1, 2, 3)]),
    }[name]
    beside_queued_work(call, sizes)


def test_calls_on_host_tensors_on_two_streams_have_workspaces_of_their_own():
    """The same shape with two filters, in turn on two streams without waits between them."""
    from gated_causal_fir_b200 import _HOST_WS
    q, k, v = (torch.randn(1, 4096, 512).to(BF16).pin_memory() for _ in range(3))
    hs = [(torch.randn(8, 128) / 11).pin_memory() for _ in range(2)]
    want = []
    for h in hs:
        want.append(g.hyena_conv_fwd_from_host(q, k, v, h, 64, 64, chunk=512))
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    runs = []
    for _ in range(6):
        for h, s in zip(hs, streams):
            runs.append(g.hyena_conv_fwd_from_host(q, k, v, h, 64, 64, stream=s, chunk=512))
    torch.cuda.synchronize()
    for i, y in enumerate(runs):
        assert torch.equal(y, want[i % 2])
    index = torch.cuda.current_device()
    places = {_HOST_WS[(index, s.cuda_stream)].data_ptr() for s in streams}
    assert len(places) == 2
