"""Sums over many terms (needs a B200): gradients of weights over long batches of tokens.

A bf16 accumulator truncates at every 16 terms, by up to 2^-23 of what it holds.  It takes at most
2^17 terms, that is 2^13 additions to partial sums that grow evenly where all terms have one sign:
2^13 x 2^-23 / 2 = 2^-11 of the sum.  The cuts' sums are added with rounding to nearest, 2^-24 each,
and the result is rounded once, 2^-8."""
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


@pytest.mark.parametrize("M,N,K", ((1 << 20, 2048, 2048), (1 << 20, 200, 72), ((1 << 18) + 77, 520, 1000),
                                   (131072, 256, 256), (131073, 256, 256), (1 << 22, 64, 16)))
def test_weight_gradients_of_many_tokens_of_one_sign(M, N, K):
    gen = torch.Generator(device="cuda").manual_seed(M + N)
    x = torch.rand(M, K, generator=gen, device="cuda", dtype=BF16) + 0.5
    dy = torch.rand(M, N, generator=gen, device="cuda", dtype=BF16) + 0.5
    dw = torch.full((N, K), float("nan"), dtype=BF16, device="cuda")
    db = torch.empty(N, device="cuda")
    g.hyena_proj_bwd(x, torch.empty_like(dw), dy, grads=(None, dw, db))
    cols = sorted({0, 1, N // 2, N - 1})
    want = torch.zeros(len(cols), K, dtype=torch.float64, device="cuda")
    for r0 in range(0, M, 1 << 16):  # in fp64, a piece at a time
        want += dy[r0:r0 + (1 << 16), cols].double().t() @ x[r0:r0 + (1 << 16)].double()
    off = ((dw[cols].double() - want) / want).abs()
    bound = (2.0 ** -11 + 64 * 2.0 ** -24) * (1 + 2.0 ** -8) + 2.0 ** -8
    assert float(off.max()) <= bound, "relative error %.3g > %.3g" % (float(off.max()), bound)
    assert bool(dw.isfinite().all())
    total = dy.sum(0, dtype=torch.float64)
    # 128 rows, then up to 2^15 / 8 blocks, then 8 threads, added in turn: fp32, to nearest
    assert float(((db.double() - total) / total).abs().max()) <= 2.0 ** -24 * (128 + M / 1024 + 8)


def test_long_reductions_forward_with_epilogue():
    """K past 2^17: every tile is cut, and bias, activation, residual and z follow the sum."""
    M, N, K = 300, 200, (1 << 17) + 1000
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.rand(M, K, generator=gen, device="cuda", dtype=BF16) + 0.5
    w = (torch.rand(N, K, generator=gen, device="cuda", dtype=BF16) + 0.5) * 2.0 ** -17
    b = torch.randn(N, generator=gen, device="cuda")
    r = torch.randn(M, N, generator=gen, device="cuda").to(BF16)
    z = torch.empty_like(r)
    y = g.hyena_proj_fwd(x, w, b, act="silu", residual=r, z=z)
    want = torch.zeros(M, N, dtype=torch.float64, device="cuda")
    for k0 in range(0, K, 1 << 15):
        want += x[:, k0:k0 + (1 << 15)].double() @ w[:, k0:k0 + (1 << 15)].double().t()
    S = want.clone()
    want = want + b.double()
    err = 2.0 ** -11 * S + 2.0 ** -24 * want.abs()
    tol = err * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
    assert bool(((z.double() - want).abs() <= tol).all())
    out = want * torch.sigmoid(want) + r.double()
    tol = 1.13 * err + 2.0 ** -19 * (1 + want.abs()) + 2.0 ** -8 * out.abs()
    assert bool(((y.double() - out).abs() <= tol * (1 + 2.0 ** -7)).all())
