"""The projections' activations and slopes element by element, in both types, where exp overflows,
vanishes or cancels (needs a B200).

The pre-activation is a bias (the product is zero), so z is exact in either type's kernel."""
import math

import pytest
import torch

import gated_causal_fir_b200 as g

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
ACTS = ("gelu", "silu", "sigmoid", "logsigmoid")
# rows of outputs that leave by TMA (bf16), by 16-byte vectors, and by single elements
WIDTHS = (1024, 1021)


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from gated_causal_fir_b200 import build
    build.build()
    g.hyena_device_status(clear=True)
    yield
    assert g.hyena_device_status(clear=True) == 0, "a kernel raised its device status word"


def forward(vals, act, dtype):
    """act(vals) of fp32 vals [N], by a projection of zeros with vals as its bias."""
    n = vals.numel()
    return g.hyena_proj_fwd(torch.zeros(1, 8, dtype=dtype, device="cuda"),
                            torch.zeros(n, 8, dtype=dtype, device="cuda"), vals, act=act)[0]


@pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "f32"))
@pytest.mark.parametrize("n", WIDTHS)
def test_infinite_values_go_to_the_limits(n, dtype):
    """+inf for every activation, -inf where the limit is no product of infinity and zero, among
    finite values; and NaN stays NaN."""
    inf = math.inf
    vals = torch.zeros(n, device="cuda")
    vals[3], vals[n - 2], vals[7] = inf, inf, math.nan
    for act, limit in (("gelu", inf), ("silu", inf), ("sigmoid", 1.0), ("logsigmoid", 0.0)):
        y = forward(vals, act, dtype)
        assert float(y[3]) == limit and float(y[n - 2]) == limit, (act, y[3], y[n - 2])
        assert bool(y[7].isnan()), act
        assert bool(y[torch.isfinite(vals)].isfinite().all()), act
    vals[3] = vals[n - 2] = -inf
    for act, limit in (("sigmoid", 0.0), ("logsigmoid", -inf)):
        y = forward(vals, act, dtype)
        assert float(y[3]) == limit and float(y[n - 2]) == limit, (act, y[3], y[n - 2])
    # a residual is added to the limit
    vals[3] = inf
    r = torch.ones(1, n, dtype=dtype, device="cuda")
    y = g.hyena_proj_fwd(torch.zeros(1, 8, dtype=dtype, device="cuda"),
                         torch.zeros(n, 8, dtype=dtype, device="cuda"), vals, act="gelu",
                         residual=r)[0]
    assert float(y[3]) == inf and float(y[0]) == 1.0
