"""The projections (hyena_proj_*) against fp64 products (needs a B200).

Bounds, with u = 2^-24 and S = |x| |w|^T.  A tensor-core product adds 16 terms to its fp32
accumulator at a time, truncating: at most 2 u of a partial sum, itself at most S, for each of the
K / 16 steps; cut products add at most 16 partial sums (u each).  fp32 operands go through six bf16
products whose smaller five are 2^-8 of S, and leave out 2^-24 S.  So |z error| <= 2 u (1.1 K / 16
+ 18) S + u |z|.  The activations' slope is at most 1.13; their own error is that of the exp they
call, 2^-21 (1 + |z|) of at most 1 with the fast exp that bf16 uses, and erf's, below it; doubled.
dz carries its slope's error and, as an operand, half a step of its type.  The last rounding is half
a step of the type."""
import math

import pytest
import torch

import gated_causal_fir_b200 as g

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
HALF = {BF16: 2.0 ** -8, F32: U}
ACTS = ("none", "gelu", "silu", "sigmoid", "logsigmoid")


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from gated_causal_fir_b200 import build
    build.build()
    g.hyena_device_status(clear=True)
    yield
    assert g.hyena_device_status(clear=True) == 0, "a kernel raised its device status word"


def act64(z, act):
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(-z * math.sqrt(0.5))
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "sigmoid":
        return torch.sigmoid(z)
    if act == "logsigmoid":
        return torch.nn.functional.logsigmoid(z)
    return z


def make(M, N, K, dtype, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed * 31 + M + 7 * N + 13 * K)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    return (r(M, K).to(dtype), (2 * r(N, K) / math.sqrt(K)).to(dtype), r(N), r(M, N).to(dtype),
            r(M, N).to(dtype))


def product_error(a, b, K):
    """Bound on the error of a b^T (fp64 operands as the tensor cores take them)."""
    return 2 * U * (1.1 * K / 16 + 18) * (a.abs() @ b.abs().t())


def within(name, got, want, err):
    assert got.shape == want.shape, name
    tol = err * (1 + HALF[got.dtype]) + HALF[got.dtype] * want.abs() + 1e-37
    d = (got.double() - want).abs()
    bad = ~(d <= tol)
    assert not bad.any(), "%s: %d of %d out of bounds, worst error/bound %.3g, first at %s" % (
        name, int(bad.sum()), bad.numel(), float((d / tol)[bad].max()), bad.nonzero()[0].tolist())


def check_forward(M, N, K, act, dtype, bias=True, residual=True, seed=0):
    x, w, b, r, _ = make(M, N, K, dtype, seed)
    b, r = (b if bias else None), (r if residual else None)
    z = torch.full((M, N), float("nan"), dtype=dtype, device="cuda")
    y = g.hyena_proj_fwd(x, w, b, act=act, residual=r, z=z)
    xd, wd = x.double(), w.double()
    want = xd @ wd.t()
    if bias:
        want = want + b.double()
    err = product_error(xd, wd, K) + U * want.abs()
    within("z", z, want, err)
    fast = 2.0 ** -20 if dtype == BF16 else 2.0 ** -21
    out = act64(want, act)
    err = 1.13 * err + (0 if act == "none" else fast * (1 + want.abs()))
    if residual:
        out = out + r.double()
    within("y", y, out, err + U * out.abs())
    return x, w, b, r, y


def check_backward(M, N, K, act, dtype, add=True, seed=0):
    x, w, b, _, dy = make(M, N, K, dtype, seed)
    z = None
    dz = dy.double()
    edz = torch.zeros_like(dz)
    if act != "none":
        z = (x.float() @ w.float().t() + b).to(dtype)
        zd = z.double().requires_grad_()
        slope, = torch.autograd.grad(act64(zd, act).sum(), zd)
        edz = dz.abs() * (2.0 ** -19 if dtype == BF16 else 2.0 ** -20) * (1 + z.double().abs())
        dz = dz * slope
    extra = torch.randn_like(x) if add else None
    dx, dw, db = g.hyena_proj_bwd(x, w, dy, z=z, act=act, dx_add=extra)
    within("db", db, dz.sum(0),
           edz.sum(0) + U * (48 + M / 1024) * (dz.abs() + edz).sum(0))
    xd, wd = x.double(), w.double()
    if act != "none":
        edz = edz + HALF[dtype] * dz.abs()
    want = dz @ wd
    err = edz @ wd.abs() + product_error(dz.abs() + edz, wd.t(), N)
    if add:
        want = want + extra.double()
    within("dx", dx, want, err + U * want.abs())
    within("dw", dw, dz.t() @ xd,
           edz.t() @ xd.abs() + product_error((dz.abs() + edz).t(), xd.t(), M))


# the smallest, single rows, ragged in each direction and around tiles, long reductions, and sizes
# for the wide tiles of CTA pairs
SHAPES = [(1, 1, 1), (1, 8, 8), (2, 16, 24), (8, 300, 4096), (1, 2048, 2048), (17, 64, 64),
          (127, 72, 65), (129, 129, 129), (128, 64, 64), (300, 515, 77), (1000, 200, 1024),
          (255, 256, 1000), (513, 1024, 512), (3000, 72, 1024), (4097, 64, 16), (64, 4097, 128)]
WIDE = [(2048, 2048, 512), (4100, 4000, 264), (2560, 4096, 1000), (2000, 4097, 130)]


@pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "f32"))
@pytest.mark.parametrize("shape", SHAPES + WIDE, ids=["x".join(map(str, s)) for s in SHAPES + WIDE])
def test_forward(shape, dtype):
    i = (SHAPES + WIDE).index(shape)
    check_forward(*shape, ACTS[i % 5], dtype, bias=i % 3 != 0, residual=i % 2 == 0)


@pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "f32"))
@pytest.mark.parametrize("shape", SHAPES + WIDE, ids=["x".join(map(str, s)) for s in SHAPES + WIDE])
def test_backward(shape, dtype):
    i = (SHAPES + WIDE).index(shape)
    check_backward(*shape, ACTS[(i + 2) % 5], dtype, add=i % 2 == 0)


@pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "f32"))
@pytest.mark.parametrize("act", ACTS)
def test_every_activation(act, dtype):
    check_forward(96, 136, 200, act, dtype)
    check_backward(96, 136, 200, act, dtype)


@pytest.mark.parametrize("act", ACTS[1:])
def test_activations_far_from_zero(act):
    """Pre-activations up to +-1e4 and infinite: the activation and its slope stay what they are
    (no overflow of exp on the way)."""
    vals = torch.tensor([-1e4, -200.0, -90.0, -30.0, -1.0, 0.0, 1.0, 30.0, 90.0, 200.0, 1e4],
                        dtype=F32, device="cuda")
    n = vals.numel()
    x = torch.zeros(1, 8, device="cuda")
    w = torch.zeros(n, 8, device="cuda")
    y = g.hyena_proj_fwd(x, w, vals, act=act)
    want = act64(vals.double(), act)[None]
    within(act, y, want, 2.0 ** -21 * (1e-30 + want.abs()) + 2.0 ** -21 * (vals.abs() < 50))
    z = vals[None].clone()
    dy = torch.ones_like(z)
    db = g.hyena_proj_bwd(x, w, dy, z=z, act=act)[2]
    zd = vals.double().requires_grad_()
    slope, = torch.autograd.grad(act64(zd, act).sum(), zd)
    within(act + " slope", db, slope, 2.0 ** -20 * (1 + vals.double().abs().clamp(max=50)))


def test_fp32_operands_of_any_size():
    """Entries from 1e-30 to 3.4e38 (where the nearest bf16 would overflow), each alone in its row
    and column: the planes give fp32's own value back."""
    vals = torch.tensor([1e-30, -3.3e-12, 0.1, 1 / 3, 12345.678, 8.5e30, 3.4e38, -3.402e38],
                        dtype=F32, device="cuda")
    x = torch.diag(vals)
    y = g.hyena_proj_fwd(x, torch.eye(8, device="cuda"))
    assert torch.equal(torch.diag(y), vals) and int((y != 0).sum()) == 8


def test_integers_are_exact():
    """Small integers: every product and partial sum is exact, so any correct order gives the same
    bits, at the edges of tiles too."""
    for M, N, K in ((130, 70, 100), (2050, 2056, 136), (9, 520, 2048)):
        gen = torch.Generator(device="cuda").manual_seed(M)
        x = torch.randint(-2, 3, (M, K), generator=gen, device="cuda").to(BF16)
        w = torch.randint(-2, 3, (N, K), generator=gen, device="cuda").to(BF16)
        dy = torch.randint(-2, 3, (M, N), generator=gen, device="cuda").to(BF16)
        y = g.hyena_proj_fwd(x, w)
        dx, dw, db = g.hyena_proj_bwd(x, w, dy)
        assert torch.equal(y, (x.double() @ w.double().t()).to(BF16))
        assert torch.equal(dx, (dy.double() @ w.double()).to(BF16))
        assert torch.equal(dw, (dy.double().t() @ x.double()).to(BF16))
        assert torch.equal(db, dy.double().sum(0).float())


def test_in_place_residual_and_wanted_gradients_only():
    x, w, b, r, dy = make(200, 96, 128, BF16)
    want = g.hyena_proj_fwd(x, w, b, act="silu", residual=r)
    y = r.clone()
    assert g.hyena_proj_fwd(x, w, b, act="silu", residual=y, y=y) is y and torch.equal(y, want)
    add = torch.randn_like(x)
    dx, dw, db = g.hyena_proj_bwd(x, w, dy, dx_add=add)
    acc = add.clone()
    assert torch.equal(g.hyena_proj_bwd(x, w, dy, dx_add=acc, grads=(acc, None, None))[0], dx)
    only = torch.empty_like(w)
    assert torch.equal(g.hyena_proj_bwd(x, w, dy, grads=(None, only, None))[1], dw)
    alone = torch.empty_like(db)
    assert torch.equal(g.hyena_proj_bwd(x, w, dy, grads=(None, None, alone))[2], db)


def test_batched_inputs_same_bits_and_bounds():
    x, w, b, r, dy = make(7 * 90, 200, 264, BF16)
    y = g.hyena_proj_fwd(x, w, b, residual=r)
    y3 = g.hyena_proj_fwd(x.view(7, 90, 264), w, b, residual=r.view(7, 90, 200))
    assert y3.shape == (7, 90, 200) and torch.equal(y3.view_as(y), y)
    buf = torch.full((y.numel() + 4096,), 7.0, dtype=BF16, device="cuda")
    for _ in range(3):
        got = g.hyena_proj_fwd(x, w, b, residual=r, y=buf[:y.numel()].view_as(y))
        assert torch.equal(got, y)
    assert (buf[y.numel():] == 7.0).all()


def test_streams_and_captured_graphs():
    M, N, K = 700, 264, 520
    x, w, b, r, dy = make(M, N, K, BF16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = g.hyena_proj_fwd(x, w, b, residual=r, stream=side)
    side.synchronize()
    assert torch.equal(y, g.hyena_proj_fwd(x, w, b, residual=r))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z = torch.empty_like(r)
        y = g.hyena_proj_fwd(x, w, b, act="gelu", residual=r, z=z)
        grads = g.hyena_proj_bwd(x, w, dy, z=z, act="gelu")
    for seed in (1, 2):
        for old, new in zip((x, w, b, r, dy), make(M, N, K, BF16, seed)):
            old.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        z2 = torch.empty_like(r)
        assert torch.equal(y, g.hyena_proj_fwd(x, w, b, act="gelu", residual=r, z=z2))
        assert torch.equal(z, z2)
        for a, c in zip(grads, g.hyena_proj_bwd(x, w, dy, z=z2, act="gelu")):
            assert torch.equal(a, c)


def test_gradient_against_differences_of_the_forward():
    """fp32, one direction per input, central differences of the forward (h = 2^-7: the third
    derivative of silu leaves h^2 / 6 ~ 1e-5 of terms like the slope's own)."""
    x, w, b, _, dy = make(60, 40, 72, F32, seed=3)
    z = torch.empty(60, 40, device="cuda")
    g.hyena_proj_fwd(x, w, b, act="silu", z=z)
    grads = g.hyena_proj_bwd(x, w, dy, z=z, act="silu")
    args, h = [x, w, b], 2.0 ** -7
    for i in range(3):
        way = torch.randn_like(args[i])
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + h * way, args[i] - h * way
        loss = [float((g.hyena_proj_fwd(*a, act="silu").double() * dy.double()).sum())
                for a in (up, down)]
        want = float((grads[i].double() * way.double()).sum())
        size = float((grads[i].double() * way.double()).abs().sum())
        assert abs((loss[0] - loss[1]) / (2 * h) - want) <= 2e-4 * size


def test_no_rows():
    x, w, b, r, dy = make(8, 24, 40, BF16)
    e = x[:0]
    assert g.hyena_proj_fwd(e, w, b).shape == (0, 24)
    dx, dw, db = g.hyena_proj_bwd(e, w, dy[:0])
    assert dx.shape == (0, 40) and not dw.any() and not db.any()


def test_refusals():
    x, w, b, r, dy = make(16, 24, 40, BF16)
    with pytest.raises(ValueError):
        g.hyena_proj_fwd(x, w, b, act="relu6")
    with pytest.raises(ValueError):
        g.hyena_proj_fwd(x, w[:, :32].contiguous(), b)
    with pytest.raises(ValueError):
        g.hyena_proj_fwd(x.t().contiguous().t(), w, b)
    with pytest.raises(TypeError):
        g.hyena_proj_fwd(x, w.float(), b)
    with pytest.raises(TypeError):
        g.hyena_proj_fwd(x, w, b.to(BF16))
    with pytest.raises(TypeError):
        g.hyena_proj_fwd(x.cpu(), w, b)
    with pytest.raises(ValueError):
        g.hyena_proj_bwd(x, w, dy, act="silu")
    with pytest.raises(ValueError):
        g.hyena_proj_fwd(x, w, residual=r[:8])
    with pytest.raises(g.HyenaError):  # 16-byte alignment
        flat = torch.empty(16 * 40 + 1, dtype=BF16, device="cuda")
        g.hyena_proj_fwd(flat[1:].view(16, 40), w, b)
    with pytest.raises(g.HyenaError):  # an output over an operand
        g.hyena_proj_bwd(x, w, dy, grads=(x, None, None))
