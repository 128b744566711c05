"""The mixer operators at the ends of their documented ranges (needs a B200)."""
import pytest
import torch

import gated_causal_fir_b200 as g
from tests import _scan_ref as R
from tests.test_mixer_gpu import make as make_layer
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


def integers(*shape, seed=0, lo=-2, hi=3):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(lo, hi, shape, generator=gen, device="cuda").to(BF16)


def test_most_rows_that_a_projections_backward_takes():
    """M = 8388480, the last whose row blocks fit a launch; small integers, so that sums are exact.
    One row more is refused."""
    M, N, K = 8388480, 8, 16
    x, w, dy = integers(M, K), integers(N, K, seed=1), integers(M, N, seed=2)
    dx, dw, db = g.hyena_proj_bwd(x, w, dy)
    assert torch.equal(db, dy.sum(0, dtype=torch.float64).float())
    want = sum(dy[r:r + (1 << 20)].double().t() @ x[r:r + (1 << 20)].double()
               for r in range(0, M, 1 << 20))
    assert torch.equal(dw, want.to(BF16))
    for r in (0, M - 5000):
        assert torch.equal(dx[r:r + 5000], (dy[r:r + 5000].double() @ w.double()).to(BF16))
    z = torch.zeros(M, N, dtype=BF16, device="cuda")
    # sigmoid'(0) = 1/4: dz is exact too
    _, dw4, db4 = g.hyena_proj_bwd(x, w, dy, z=z, act="sigmoid", grads=(None, dw.clone(), db.clone()))
    assert torch.equal(db4, db / 4) and torch.equal(dw4, (want / 4).to(BF16))
    del dx, z
    with pytest.raises(g.HyenaError):
        g.hyena_proj_bwd(torch.empty(M + 1, K, dtype=BF16, device="cuda"), w,
                         torch.empty(M + 1, N, dtype=BF16, device="cuda"))


@pytest.mark.parametrize("M,N,K", ((1 << 22, 1, 1), (3, 1 << 20, 8), (1, 5, 1 << 20),
                                   (2, 3, 1 << 24), (1 << 20, 9, 3)))
def test_long_and_thin_projections(M, N, K):
    x, w = integers(M, K, lo=0, hi=2), integers(N, K, seed=1, lo=0, hi=2)
    y = g.hyena_proj_fwd(x, w)
    r = slice(0, M) if M < 4096 else slice(M - 4096, M)
    want = torch.zeros(x[r].shape[0], N, dtype=torch.float64, device="cuda")
    for k in range(0, K, 1 << 20):
        want += x[r, k:k + (1 << 20)].double() @ w[:, k:k + (1 << 20)].double().t()
    assert torch.equal(y[r], want.to(BF16))  # sums of ones are exact


@pytest.mark.parametrize("B,L,D,d_g", ((70000, 1, 8, 1), (3000, 5, 40, 8), (1, 1, 65536, 64)))
def test_many_short_sequences(B, L, D, d_g):
    q, k, v, lg, s0, dy, ds = make(B, L, D, d_g, BF16)
    ref = R.Ref(q, k, v, lg, d_g, s0, dy, ds)
    y, s_out = g.hyena_scan_fwd(q, k, v, lg, d_g, s0=s0)
    R.check("y", y, ref)
    R.check("s_out", s_out, ref)
    for name, t in zip(("dq", "dk", "dv", "dg", "ds0"),
                       g.hyena_scan_bwd(q, k, v, lg, dy, d_g, s0=s0, ds_out=ds)):
        R.check(name, t, ref)


@pytest.mark.parametrize("kind", ("scan", "fir"))
@pytest.mark.parametrize("B,L", ((0, 5), (2, 0)))
def test_layers_of_no_tokens(kind, B, L):
    p = make_layer(kind, 64, 64, 16, BF16)
    x = torch.zeros(B, L, 64, dtype=BF16, device="cuda")
    out, state, saved = g.hyena_mixer_fwd(x, p, save=True)
    assert out.shape == x.shape and (kind == "fir" or not state.any())
    dx, ds0, grads = g.hyena_mixer_bwd(x, p, saved, x)
    assert dx.shape == x.shape
    for n, d in grads.items():
        for t in (d if isinstance(d, tuple) else (d,)):
            assert not t.any(), n


def test_the_same_tensor_for_several_inputs():
    """q, k and v one tensor; x its own residual; dy also as dx_add."""
    q, _, _, lg, s0, _, ds = make(2, 300, 64, 16, BF16)
    ref = R.Ref(q, q, q, lg, 16, s0, q, ds)
    y, _ = g.hyena_scan_fwd(q, q, q, lg, 16, s0=s0)
    R.check("y", y, ref)
    for name, t in zip(("dq", "dk", "dv", "dg", "ds0"),
                       g.hyena_scan_bwd(q, q, q, lg, q, 16, s0=s0, ds_out=ds)):
        R.check(name, t, ref)
    x, w = integers(300, 64), integers(64, 64, seed=3)
    assert torch.equal(g.hyena_proj_fwd(x, w, residual=x),
                       (x.double() @ w.double().t() + x.double()).to(BF16))
    dx, dw, _ = g.hyena_proj_bwd(x, w, x, dx_add=x)
    assert torch.equal(dx, (x.double() @ w.double() + x.double()).to(BF16))
    assert torch.equal(dw, (x.double().t() @ x.double()).to(BF16))
