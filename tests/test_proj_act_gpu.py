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


# Relative bounds, with u = 2^-24 and the errors that CUDA's documentation gives (fp32: expf 2 ulp,
# erfcf 4, log1pf 1; fast forms: __expf 2 + floor(|1.173 z|) ulp, __fdividef 2, __logf 2^-21.41
# absolute on [0.5, 2]; an ulp is at most 2 u of the value).
#   phi      erfc's argument carries 2 roundings, which z^2 + 1 times as much of erfc answers for:
#            8 u + 2 (z^2 + 1) u; bf16: 2^-12 of the fit, 3e-7 of 1 where Phi is near 1, and the
#            exponential's ulps and its argument's half a rounding of z^2 / 2
#   sigmoid  the exponential's ulps, the division, two or three roundings
# doubled.  A bf16 result is rounded once more, by half a step.
U = 2.0 ** -24


def phi64(z):
    return 0.5 * torch.special.erfc(-z * math.sqrt(0.5))


def rel_of(z, dtype):
    """Relative errors of (Phi, exp and what is made of it)."""
    if dtype == F32:
        return 2 * U * (10 + 2 * (z * z + 1)), 2 * U * (12 + 0 * z)
    ulps = lambda x: 2 * U * (2 * (2 + 1.173 * x) + 8)  # noqa: E731
    return 2 * (2.0 ** -12 + 2 * 3e-7) + ulps(z * z / 2) + 2 * U * z * z, ulps(z.abs())


def definition(z, act, dtype):
    """(value, error bound before the last rounding) in fp64."""
    phi, rel = rel_of(z, dtype)
    if act == "gelu":
        v = z * phi64(z)
        return v, v.abs() * (phi + U)
    s = torch.sigmoid(z)
    if act == "silu":
        return z * s, (z * s).abs() * rel
    if act == "sigmoid":
        return s, s * rel
    v = torch.where(z > 0, -torch.log1p(torch.exp(-z)), torch.nn.functional.logsigmoid(z))
    # log(1 + e) of bf16 results: the series below e = 2^-6 (2^-20), else 2^-21.41 of at least 2^-6.1
    return v, v.abs() * (rel + (0 if dtype == F32 else 2.0 ** -15))


def slope_definition(z, act, dtype):
    phi, rel = rel_of(z, dtype)
    if act == "gelu":
        a, b = phi64(z), z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
        return a + b, a * phi + b.abs() * (phi if dtype == BF16 else rel + 2 * U * (2 + z * z))
    p, m = torch.sigmoid(z), torch.sigmoid(-z)
    if act == "silu":  # p (1 + z m); m is 1 - p, with an error of u where p is near 1
        return p * (1 + z * m), p * (1 + z.abs() * m) * 2 * rel + 2 * U * p * z.abs()
    if act == "sigmoid":
        return p * m, p * m * 2 * rel
    return m, m * rel


def near(name, got, want, err):
    half = {BF16: 2.0 ** -8, F32: U}[got.dtype]
    tol = err * (1 + half) + half * want.abs() + 1e-37
    off = (got.double() - want).abs() / tol
    assert float(off.max()) <= 1.0, "%s: error/bound %.3g at %d" % (name, float(off.max()),
                                                                   int(off.argmax()))


@pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "f32"))
@pytest.mark.parametrize("act", ACTS)
def test_tails_keep_their_bits(act, dtype):
    """z from -12 to 20, where the values fall to 1e-32: errors relative to the value, not to 1."""
    for n in WIDTHS:
        vals = torch.linspace(-12, 20, n, device="cuda")
        near(act, forward(vals, act, dtype), *definition(vals.double(), act, dtype))
        z = vals.to(dtype)[None]
        slope = g.hyena_proj_bwd(torch.zeros(1, 8, dtype=dtype, device="cuda"),
                                 torch.zeros(n, 8, dtype=dtype, device="cuda"),
                                 torch.ones_like(z), z=z, act=act)[2]
        near(act + " slope", slope, *slope_definition(z[0].double(), act, dtype))


def test_fp32_operands_down_to_the_smallest():
    """Operands of every size against partners that bring their products back to ordinary ones.  At
    2^-110 and above the three planes hold all 24 bits; below, bf16's last bit 2^-133 leaves an error
    of half of it (2^-134) in the operand.  The bound is the products' own (test_proj_gpu: 2 u (1.1 K
    / 16 + 18) S) and 2^-133 of the partner."""
    small = torch.tensor([2.0 ** -100, 1.2345678 * 2.0 ** -109, (1 + 2.0 ** -23) * 2.0 ** -110,
                          1.7654321 * 2.0 ** -111, 1.0001e-34, 3.3333333e-36, 1.0001e-38,
                          1.1754945e-38, 5.4321e-39, 2.0 ** -133, 2.0 ** -140, 0.0],
                         dtype=torch.float64).float().cuda()
    big = torch.tensor([3.4e38, 2.0 ** 100, 1.5, -2.2222222e37], device="cuda")
    n = small.numel()
    w = torch.zeros(n, 8, device="cuda")
    w[:, 3] = small
    for b in big:
        x = torch.zeros(5, 8, device="cuda")
        x[:, 3] = b
        y = g.hyena_proj_fwd(x, w)[0].double()
        want = float(b) * small.double()
        lost = torch.where(small.double().abs() >= 2.0 ** -110, 0.0, 2.0 ** -133) * abs(float(b))
        err = 2 * U * (1.1 * 8 / 16 + 18) * want.abs() + lost
        # results below fp32's normal numbers keep fewer bits
        assert bool(((y - want).abs() <= err + U * want.abs() + 2.0 ** -126).all()), (float(b), y, want)
