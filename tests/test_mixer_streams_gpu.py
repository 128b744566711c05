"""Calls on a stream that the caller gives, beside work on the current one that they do not wait for
(needs a B200).

What such a call makes for itself or returns must not be memory that queued work on the current
stream still uses: freed there, it is the caching allocator's first choice for the current stream."""
import pytest
import torch

import gated_causal_fir_b200 as g

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from gated_causal_fir_b200 import build
    build.build()
    g.hyena_device_status(clear=True)
    yield
    assert g.hyena_device_status(clear=True) == 0, "a kernel raised its device status word"


def calls():
    """{name: (call(stream), sizes in bytes of what it makes)} over inputs that are ready."""
    rand = lambda *s, dtype=BF16: torch.randn(*s, device="cuda").to(dtype)  # noqa: E731
    out = {}
    # the time axis cut (workspace), fp32 states
    B, L, D, d_g = 1, 20000, 64, 64
    q, k, v, dy = (rand(B, L, D) for _ in range(4))
    lg = -torch.rand(B, L, 1, device="cuda").to(BF16)
    sizes = [q.numel() * 2, lg.numel() * 2, D * 4,
             g.hyena_scan_workspace_bytes(B, L, D, d_g),
             g.hyena_scan_bwd_workspace_bytes(B, L, D, d_g, have_ckpt=False)]
    out["scan_fwd"] = (lambda s: g.hyena_scan_fwd(q, k, v, lg, d_g, stream=s), sizes)
    out["scan_bwd"] = (lambda s: g.hyena_scan_bwd(q, k, v, lg, dy, d_g, stream=s), sizes)
    state, advanced = rand(512, 64, dtype=F32), rand(512, 64, dtype=F32)
    one = [rand(512, 64) for _ in range(3)] + [-torch.rand(512, 1, device="cuda").to(BF16)]
    out["scan_step"] = (lambda s: g.hyena_scan_step(*one, state, 64,
                                                    state_out=advanced, stream=s)[0],
                        [512 * 64 * 2])
    # fp32 operands are packed into the workspace
    x, w, z = rand(700, 300, dtype=F32), rand(200, 300, dtype=F32), rand(700, 200, dtype=F32)
    out["proj_fwd"] = (lambda s: g.hyena_proj_fwd(x, w, act="silu", stream=s),
                       [z.numel() * 4, g.hyena_proj_workspace_bytes(700, 200, 300,
                                                                    g.HYENA_DTYPE_F32)])
    out["proj_bwd"] = (lambda s: g.hyena_proj_bwd(x, w, z, z=z, act="silu", stream=s),
                       [x.numel() * 4, w.numel() * 4, 800,
                        g.hyena_proj_bwd_workspace_bytes(700, 200, 300, "silu",
                                                         g.HYENA_DTYPE_F32)])
    return out


NAMES = ("scan_fwd", "scan_bwd", "scan_step", "proj_fwd", "proj_bwd")


def tensors(r):
    return [r] if isinstance(r, torch.Tensor) else list(r)


def beside_queued_work(call, sizes):
    """The call's results on another stream while the current one still has to write to blocks of
    the sizes that the call makes, freed a moment before; they are what they are alone."""
    side = torch.cuda.Stream()
    want = [t.clone() for t in tensors(call(None))]
    torch.cuda.synchronize()
    for _ in range(3):
        torch.cuda._sleep(100_000_000)  # about 50 ms
        blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
        for b in blocks:
            b.fill_(0x7f)
        places = [(b.data_ptr(), b.data_ptr() + b.numel()) for b in blocks]
        del blocks, b
        got = tensors(call(side))
        for t in got:
            assert not any(lo <= t.data_ptr() < hi for lo, hi in places), \
                "a result lies in memory that the current stream is about to write"
        torch.cuda.synchronize()  # the queued writes have happened
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        del got, a, b


@pytest.mark.parametrize("name", NAMES)
def test_a_given_stream_does_not_share_freed_memory_with_the_current_one(name):
    beside_queued_work(*calls()[name])


@pytest.mark.parametrize("name", NAMES)
def test_a_result_dropped_on_the_current_stream_is_not_reused_under_its_reader(name):
    """A result read by queued work of the current stream and dropped: the next call on the given
    stream must not take its memory before that work is done."""
    call, _ = calls()[name]
    side, main = torch.cuda.Stream(), torch.cuda.current_stream()
    want = [t.clone() for t in tensors(call(None))]
    torch.cuda.synchronize()
    got = tensors(call(side))
    main.wait_stream(side)
    torch.cuda._sleep(100_000_000)
    copies = [t.clone() for t in got]  # queued behind the sleep
    del got
    for _ in range(4):  # would take the dropped results' memory
        call(side)
        filler = [torch.empty_like(t) for t in copies]
        with torch.cuda.stream(side):
            for t in copies:
                torch.empty_like(t).fill_(0)
        del filler
    torch.cuda.synchronize()
    for a, b in zip(copies, want):
        assert torch.equal(a, b)
