"""The forward as inference calls it (needs a B200): bias, activation and residual without the value
before the activation, whose epilogue, where whole bf16 tiles leave by TMA and residuals arrive by
it, no call that keeps z takes.  Bounds: test_proj_gpu."""
import math

import pytest
import torch

import gated_causal_fir_b200 as g
from tests.test_proj_act_gpu import definition, forward, near, slope_definition
from tests.test_proj_gpu import ACTS, SHAPES, U, WIDE, act64, make, product_error, within

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


# beside those of test_proj_gpu: whole waves of 128-wide tiles, waves with a cut rest, single tiles
MORE = [(128, 128, 64), (4736, 512, 64), (5000, 1024, 2048), (9472, 512, 2048), (600, 8, 8)]
ALL = SHAPES + WIDE + MORE


def check(M, N, K, act, dtype, bias, residual, seed=0, in_place=False):
    x, w, b, r, _ = make(M, N, K, dtype, seed)
    b, r = (b if bias else None), (r if residual else None)
    want = x.double() @ w.double().t()
    if bias:
        want = want + b.double()
    err = product_error(x.double(), w.double(), K) + U * want.abs()
    fast = 2.0 ** -20 if dtype == BF16 else 2.0 ** -21
    out = act64(want, act)
    err = 1.13 * err + (0 if act == "none" else fast * (1 + want.abs()))
    if residual:
        out = out + r.double()
    y = r if in_place else torch.full((M, N), float("nan"), dtype=dtype, device="cuda")
    y = g.hyena_proj_fwd(x, w, b, act=act, residual=r, y=y)
    within("y", y, out, err + U * out.abs())


@pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "f32"))
@pytest.mark.parametrize("shape", ALL, ids=["x".join(map(str, s)) for s in ALL])
def test_bias_activation_and_residual(shape, dtype):
    i = ALL.index(shape)
    check(*shape, ACTS[i % 5], dtype, True, True, seed=2)
    check(*shape, ACTS[(i + 1) % 5], dtype, i % 2 == 0, True, seed=3, in_place=True)
    check(*shape, ACTS[(i + 3) % 5], dtype, True, False, seed=4)


@pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "f32"))
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("shape", ((1100, 264, 72), (4736, 512, 64), (2048, 2048, 512)),
                         ids=lambda s: "x".join(map(str, s)))
def test_every_activation_with_bias_and_residual(shape, act, dtype):
    for bias in (True, False):
        check(*shape, act, dtype, bias, True, seed=5)


@pytest.mark.parametrize("act", ACTS[1:])
@pytest.mark.parametrize("n", (1024, 1021))
def test_bf16_far_from_zero(n, act):
    """Where exp overflows or vanishes; relative bounds as for the tails, and 1e-37."""
    far = torch.tensor([-1e30, -1e4, -200.0, -90.0, -87.0, -60.0, -13.0, 21.0, 60.0, 87.0, 90.0,
                        200.0, 1e4, 1e30], device="cuda")
    vals = far.repeat(n // far.numel() + 1)[:n].contiguous()
    want, err = definition(vals.double(), act, BF16)
    near(act, forward(vals, act, BF16), want, torch.nan_to_num(err, posinf=0.0).clamp(
        max=2.0 ** -6 * want.abs() + 1e-37))
    z = vals.to(BF16)[None]
    slope = g.hyena_proj_bwd(torch.zeros(1, 8, dtype=BF16, device="cuda"),
                             torch.zeros(n, 8, dtype=BF16, device="cuda"), torch.ones_like(z), z=z,
                             act=act)[2]
    want, err = slope_definition(z[0].double(), act, BF16)
    near(act + " slope", slope, want, torch.nan_to_num(err, posinf=0.0).clamp(
        max=2.0 ** -6 * want.abs() + 1e-37))
    assert math.isfinite(float(slope.sum()))
