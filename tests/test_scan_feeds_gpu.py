"""The recurrence where its streams and its groups' rows reach shared memory in different ways, and
where it is called again and again (needs a B200).  Bounds: _scan_ref."""
import pytest
import torch

import gated_causal_fir_b200 as g
from tests import _scan_ref as R
from tests.test_scan_gpu import make

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


def moved(t, elements):
    """The values of t in a contiguous view that starts `elements` into its storage."""
    base = torch.empty(t.numel() + elements, dtype=t.dtype, device=t.device)
    base[elements:] = t.flatten()
    return base[elements:].view(t.shape)


@pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "f32"))
@pytest.mark.parametrize("B,L,D,d_g,shift", (
    (1, 700, 24, 3, 0), (2, 900, 72, 9, 0), (1, 2500, 40, 5, 0), (1, 20000, 56, 7, 0),
    (2, 400, 200, 25, 0),        # odd groups: TMA cannot give a pair of channels one decay
    (1, 700, 128, 16, 4), (1, 900, 128, 16, 2), (2, 500, 2048, 64, 4)))  # streams off 16 bytes
def test_copied_streams_with_groups_rows_that_tma_could_take(B, L, D, d_g, shift, dtype):
    """q, k, v, dy arrive by asynchronous copies while the groups' rows (whole 16-byte vectors, in
    aligned memory) are stored by the helper threads: both are in the tile when it is read."""
    q, k, v, lg, s0, dy, ds = make(B, L, D, d_g, dtype, seed=3)
    ref = R.Ref(q, k, v, lg, d_g, s0, dy, ds)
    if shift:
        q, k, v, dy = (moved(t, shift) for t in (q, k, v, dy))
    first = None
    for _ in range(8):
        ckpt = g.hyena_scan_ckpt(q)
        y, s_out = g.hyena_scan_fwd(q, k, v, lg, d_g, s0=s0, ckpt=ckpt)
        got = [y, s_out] + list(g.hyena_scan_bwd(q, k, v, lg, dy, d_g, s0=s0, ds_out=ds, ckpt=ckpt))
        if first is None:
            first = got
            for name, t in zip(("y", "s_out", "dq", "dk", "dv", "dg", "ds0"), got):
                R.check(name, t, ref)
        for a, b in zip(got, first):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "f32"))
@pytest.mark.parametrize("L,D,d_g", ((4000, 4096, 64), (4000, 4096, 1), (3000, 1032, 3),
                                     (20000, 256, 16)))
def test_tiles_are_read_before_the_next_ones_land(L, D, d_g, dtype):
    """Rings that turn over many times, called again and again over changing neighbours: the same
    bits in every call."""
    q, k, v, lg, s0, dy, ds = make(1, L, D, d_g, dtype, seed=11)
    ckpt = g.hyena_scan_ckpt(q)
    want = None
    for _ in range(30):
        y, s_out = g.hyena_scan_fwd(q, k, v, lg, d_g, s0=s0, ckpt=ckpt)
        got = [y, s_out, *g.hyena_scan_bwd(q, k, v, lg, dy, d_g, s0=s0, ds_out=ds, ckpt=ckpt)]
        if want is None:
            want = got
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "f32"))
@pytest.mark.parametrize("B,L,D", ((1, 400, 4096), (2, 1500, 128), (1, 20000, 64), (1, 333, 72),
                                   (3, 200, 240), (1, 900, 48), (1, 178, 8)))
def test_groups_of_eight(B, L, D, dtype):
    """The widest groups whose exps the forward's compute warps take: whole rows, clusters, cuts,
    groups' rows by TMA and by copies."""
    q, k, v, lg, s0, dy, ds = make(B, L, D, 8, dtype, seed=2, resets=True)
    ref = R.Ref(q, k, v, lg, 8, s0, dy, ds)
    ckpt = g.hyena_scan_ckpt(q)
    y, s_out = g.hyena_scan_fwd(q, k, v, lg, 8, s0=s0, ckpt=ckpt)
    R.check("y", y, ref)
    R.check("s_out", s_out, ref)
    grads = g.hyena_scan_bwd(q, k, v, lg, dy, 8, s0=s0, ds_out=ds, ckpt=ckpt)
    for name, t, again in zip(("dq", "dk", "dv", "dg", "ds0"), grads,
                              g.hyena_scan_bwd(q, k, v, lg, dy, 8, s0=s0, ds_out=ds)):
        R.check(name, t, ref)
        assert torch.equal(t, again)
