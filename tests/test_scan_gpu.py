"""The gated linear recurrence (hyena_scan_*) against its fp64 definition, within the bounds that
_scan_ref derives (needs a B200)."""
import math

import pytest
import torch

import gated_causal_fir_b200 as g
from tests import _scan_ref as R

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


def make(B, L, D, d_g, dtype, seed=0, resets=False):
    gen = torch.Generator().manual_seed(seed * 7919 + L + D)
    q, k, v, dy = (torch.randn(B, L, D, generator=gen).to(dtype).cuda() for _ in range(4))
    lg = -torch.exp(torch.empty(B, 1, D // d_g).uniform_(math.log(1e-3), 0.0, generator=gen) +
                    0.5 * torch.randn(B, L, D // d_g, generator=gen))
    if resets and L > 1:
        lg[torch.rand(B, L, generator=gen) < 0.05] = -math.inf
    s0, ds = (torch.randn(B, D, generator=gen).cuda() for _ in range(2))
    return q, k, v, lg.to(dtype).cuda(), s0, dy, ds


# rows of a tile: 176 (bf16), 112 (fp32)
SHAPES = [
    # B, L, D, d_g
    (1, 1, 8, 1), (2, 1, 64, 64), (1, 2, 32, 8), (3, 7, 40, 1), (1, 175, 64, 16), (1, 176, 64, 1),
    (2, 177, 64, 64), (1, 111, 96, 96), (1, 112, 128, 128), (2, 113, 72, 2), (1, 353, 200, 8),
    (2, 1000, 96, 48), (1, 700, 36, 3), (1, 401, 33, 1), (2, 333, 35, 5), (1, 260, 7, 7),
    (1, 300, 1, 1), (1, 143, 64, 4), (2, 144, 64, 2), (1, 145, 128, 32), (1, 289, 264, 4),
    (2, 300, 66, 2), (1, 700, 100, 2),
    (2, 200, 1732, 2), (1, 310, 440, 8), (1, 300, 488, 8), (1, 200, 272, 16), (2, 180, 192, 96),
    (1, 200, 208, 4), (1, 150, 24, 2), (1, 330, 50, 10),
    # clusters of 2 to 8 CTAs, with and without an empty last round; the time axis cut
    (1, 530, 96, 1), (2, 900, 64, 32), (1, 1250, 320, 64), (3, 1410, 100, 2), (1, 2500, 36, 1),
    # groups of 2 and 4 (their exps where they are used) shared by clusters and by cuts
    (1, 900, 64, 2), (2, 1500, 128, 4), (1, 20000, 64, 2), (1, 353, 2048, 2),
    (1, 1600, 512, 16), (1, 9000, 48, 48), (2, 20000, 8, 1), (1, 5000, 32, 1), (1, 4000, 72, 24), (5, 190, 1024, 1), (160, 3, 64, 32),
]


@pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "f32"))
@pytest.mark.parametrize("shape", SHAPES, ids=["x".join(map(str, s)) for s in SHAPES])
def test_forward_and_backward(shape, dtype):
    B, L, D, d_g = shape
    q, k, v, lg, s0, dy, ds = make(B, L, D, d_g, dtype, resets=L % 2 == 1)
    ref = R.Ref(q, k, v, lg, d_g, s0, dy, ds)
    ckpt = g.hyena_scan_ckpt(q)
    y, s_out = g.hyena_scan_fwd(q, k, v, lg, d_g, s0=s0, ckpt=ckpt)
    grads = g.hyena_scan_bwd(q, k, v, lg, dy, d_g, s0=s0, ds_out=ds, ckpt=ckpt)
    R.check("y", y, ref)
    R.check("s_out", s_out, ref)
    for name, t in zip(("dq", "dk", "dv", "dg", "ds0"), grads):
        R.check(name, t, ref)
    y, s_out = g.hyena_scan_fwd(q, k, v, lg, d_g, s0=s0)
    R.check("y", y, ref)
    R.check("s_out", s_out, ref)
    # without the checkpoints the states are found again, to the same bits
    again = g.hyena_scan_bwd(q, k, v, lg, dy, d_g, s0=s0, ds_out=ds)
    for a, b in zip(grads, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "f32"))
def test_no_initial_state_and_no_state_gradient(dtype):
    q, k, v, lg, _, dy, _ = make(2, 250, 96, 16, dtype)
    ref = R.Ref(q, k, v, lg, 16, None, dy, None)
    y, s_out = g.hyena_scan_fwd(q, k, v, lg, 16)
    R.check("y", y, ref)
    R.check("s_out", s_out, ref)
    for name, t in zip(("dq", "dk", "dv", "dg", "ds0"), g.hyena_scan_bwd(q, k, v, lg, dy, 16)):
        R.check(name, t, ref)


@pytest.mark.parametrize("d_g", (1, 16))
def test_unaligned_views_take_the_element_loads(d_g):
    """Contiguous views that start 2 bytes into their storage, each input in turn."""
    q, k, v, lg, s0, dy, ds = make(1, 200, 64, d_g, BF16)
    ref = R.Ref(q, k, v, lg, d_g, s0, dy, ds)

    def shifted(t):
        base = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
        base[1:] = t.flatten()
        return base[1:].view(t.shape)

    for i in range(5):
        a = [shifted(t) if i == j else t for j, t in enumerate((q, k, v, lg, dy))]
        y, s_out = g.hyena_scan_fwd(a[0], a[1], a[2], a[3], d_g, s0=s0)
        R.check("y", y, ref)
        R.check("s_out", s_out, ref)
        grads = g.hyena_scan_bwd(a[0], a[1], a[2], a[3], a[4], d_g, s0=s0, ds_out=ds)
        for name, t in zip(("dq", "dk", "dv", "dg", "ds0"), grads):
            R.check(name, t, ref)
    out = shifted(torch.zeros_like(lg))
    grads = (torch.empty_like(q), torch.empty_like(q), torch.empty_like(q), out,
             torch.empty_like(s0))
    g.hyena_scan_bwd(q, k, v, lg, dy, d_g, s0=s0, ds_out=ds, grads=grads)
    R.check("dg", out, ref)


def test_reset_forgets_and_decay_zero_keeps():
    """g = -inf: the tokens before do not count, in either direction; g = 0: the state is a sum."""
    q, k, v, lg, s0, dy, ds = make(1, 300, 64, 64, BF16)
    lg.zero_()
    lg[:, 100] = -math.inf
    ref = R.Ref(q, k, v, lg, 64, s0, dy, ds)
    y, s_out = g.hyena_scan_fwd(q, k, v, lg, 64, s0=s0)
    R.check("y", y, ref)
    R.check("s_out", s_out, ref)
    tail, t_out = g.hyena_scan_fwd(*(t[:, 100:].contiguous() for t in (q, k, v, lg)), 64)
    assert torch.allclose(t_out, s_out, rtol=0, atol=1e-4)
    grads = g.hyena_scan_bwd(q, k, v, lg, dy, 64, s0=s0, ds_out=ds)
    for name, t in zip(("dq", "dk", "dv", "dg", "ds0"), grads):
        R.check(name, t, ref)
    assert not grads[3][:, 100].any()  # exp(-inf) s = 0: no gradient through a reset


@pytest.mark.parametrize("L,D", ((1, 64), (600, 64), (4000, 40)))
def test_pieces_of_a_sequence_continue_each_other(L, D):
    q, k, v, lg, s0, dy, ds = make(2, L, D, 8, F32)
    ref = R.Ref(q, k, v, lg, 8, s0, dy, ds)
    ys, s = [], s0
    for t0, t1 in ((0, L // 3), (L // 3, L // 3), (L // 3, L)):  # an empty piece too
        y, s = g.hyena_scan_fwd(*(t[:, t0:t1].contiguous() for t in (q, k, v, lg)), 8, s0=s)
        ys.append(y)
    R.check("y", torch.cat(ys, 1), ref)
    R.check("s_out", s, ref)


@pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "f32"))
@pytest.mark.parametrize("B,D,d_g", ((1, 4096, 1), (7, 96, 48), (64, 512, 64), (3, 33, 11),
                                     (2, 40, 2), (1, 1, 1), (5, 24, 3)))
def test_step(B, D, d_g, dtype):
    q, k, v, lg, s0, _, _ = make(B, 1, D, d_g, dtype)
    ref = R.Ref(q, k, v, lg, d_g, s0)
    args = [t[:, 0].contiguous() for t in (q, k, v, lg)]
    kept = s0.clone()
    y, s = g.hyena_scan_step(*args, s0, d_g, state_out=torch.empty_like(s0))
    assert torch.equal(s0, kept)
    R.check("y", y[:, None], ref)
    R.check("s_out", s, ref)
    y2, s2 = g.hyena_scan_step(*args, s0, d_g)  # in place
    assert s2.data_ptr() == s0.data_ptr() and torch.equal(s2, s) and torch.equal(y2, y)


def test_gradient_against_differences_of_the_forward():
    """fp32, one direction per input: the forward's slope by central differences.  h = 2^-6: the
    forward is a polynomial of degree at most 2 along q, k, v, s0 (central differences exact); along
    g the third derivative leaves h^2 / 6 ~ 4e-5 of terms like the slope's own."""
    q, k, v, lg, s0, dy, ds = make(1, 200, 64, 16, F32, seed=5)
    grads = g.hyena_scan_bwd(q, k, v, lg, dy, 16, s0=s0, ds_out=ds)
    gen = torch.Generator().manual_seed(1)

    def loss(a):
        y, s = g.hyena_scan_fwd(a[0], a[1], a[2], a[3], 16, s0=a[4])
        return float((y.double() * dy.double()).sum() + (s.double() * ds.double()).sum())

    args = [q, k, v, lg, s0]
    h = 2.0 ** -6
    for i in range(5):
        way = torch.randn(args[i].shape, generator=gen).cuda()
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + h * way, args[i] - h * way
        slope = (loss(up) - loss(down)) / (2 * h)
        size = float((grads[i].double() * way.double()).abs().sum())
        assert abs(slope - float((grads[i].double() * way.double()).sum())) <= 2e-4 * size


def test_same_bits_in_every_call_and_outputs_stay_in_bounds():
    """Repeated calls give the same bits, and nothing is written past an output."""
    q, k, v, lg, s0, dy, ds = make(2, 611, 1000, 1, BF16)
    want = None
    for _ in range(5):
        ybuf = torch.full((q.numel() + 4096,), 7.0, dtype=BF16, device="cuda")
        y = ybuf[:q.numel()].view(q.shape)
        _, s_out = g.hyena_scan_fwd(q, k, v, lg, 1, s0=s0, y=y)
        got = [y, s_out] + list(g.hyena_scan_bwd(q, k, v, lg, dy, 1, s0=s0, ds_out=ds))
        torch.cuda.synchronize()
        assert (ybuf[q.numel():] == 7.0).all()
        if want is None:
            want = [t.clone() for t in got]
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_streams_and_captured_graphs():
    """A call on another stream, and captured forward, backward and step replayed on new data."""
    q, k, v, lg, s0, dy, ds = make(1, 3000, 64, 64, BF16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, s_out = g.hyena_scan_fwd(q, k, v, lg, 64, s0=s0, stream=side)
    side.synchronize()
    ref = R.Ref(q, k, v, lg, 64, s0, dy, ds)
    R.check("y", y, ref)
    R.check("s_out", s_out, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ckpt = g.hyena_scan_ckpt(q)
        y, s_out = g.hyena_scan_fwd(q, k, v, lg, 64, s0=s0, ckpt=ckpt)
        grads = g.hyena_scan_bwd(q, k, v, lg, dy, 64, s0=s0, ds_out=ds, ckpt=ckpt)
        yt, st = g.hyena_scan_step(q[:, 0], k[:, 0], v[:, 0], lg[:, 0], s_out, 64,
                                   state_out=torch.empty_like(s_out))
    for seed in (1, 2):
        new = make(1, 3000, 64, 64, BF16, seed=seed)
        for old, n in zip((q, k, v, lg, s0, dy, ds), new):
            old.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        ref = R.Ref(q, k, v, lg, 64, s0, dy, ds)
        R.check("y", y, ref)
        R.check("s_out", s_out, ref)
        for name, t in zip(("dq", "dk", "dv", "dg", "ds0"), grads):
            R.check(name, t, ref)
        one = R.Ref(q[:, :1], k[:, :1], v[:, :1], lg[:, :1], 64, s_out)
        R.check("s_out", st, one)


def test_empty_problems():
    q = torch.zeros(2, 0, 64, dtype=BF16, device="cuda")
    lg = torch.zeros(2, 0, 1, dtype=BF16, device="cuda")
    s0 = torch.randn(2, 64, device="cuda")
    y, s = g.hyena_scan_fwd(q, q, q, lg, 64, s0=s0)
    assert y.shape == q.shape and torch.equal(s, s0)
    assert not g.hyena_scan_fwd(q, q, q, lg, 64)[1].any()
    assert torch.equal(g.hyena_scan_bwd(q, q, q, lg, q, 64, ds_out=s0)[4], s0)
    none = torch.zeros(0, 5, 64, dtype=BF16, device="cuda")
    assert g.hyena_scan_fwd(none, none, none, none[..., :1].contiguous(), 64)[0].shape == none.shape


def test_refusals():
    q, k, v, lg, s0, dy, ds = make(2, 20, 64, 16, BF16)
    with pytest.raises(ValueError):  # not contiguous
        g.hyena_scan_fwd(q.transpose(0, 1).contiguous().transpose(0, 1), k, v, lg, 16)
    with pytest.raises(ValueError):
        g.hyena_scan_fwd(q, k[:, :10], v, lg, 16)
    with pytest.raises(ValueError):
        g.hyena_scan_fwd(q, k, v, lg, 24)
    with pytest.raises(ValueError):  # one decay per channel expected
        g.hyena_scan_fwd(q, k, v, lg, 1)
    with pytest.raises(TypeError):
        g.hyena_scan_fwd(q, k.float(), v, lg, 16)
    with pytest.raises(TypeError):
        g.hyena_scan_fwd(q.half(), k.half(), v.half(), lg.half(), 16)
    with pytest.raises(TypeError):
        g.hyena_scan_fwd(q, k, v, lg, 16, s0=s0.to(BF16))
    with pytest.raises(g.HyenaError):  # output over an input
        g.hyena_scan_fwd(q, k, v, lg, 16, y=q)
    with pytest.raises(g.HyenaError):  # the state is not advanced in place here
        g.hyena_scan_fwd(q, k, v, lg, 16, s0=s0, s_out=s0)
    with pytest.raises(ValueError):
        g.hyena_scan_bwd(q, k, v, lg, dy, 16, ckpt=torch.empty(2, 5, 64, device="cuda"))
    with pytest.raises(ValueError):
        g.hyena_scan_step(q[:, 0].contiguous(), k[:, 0].contiguous(), v[:, 0].contiguous(),
                          lg[:, 0].contiguous(), None, 16)
