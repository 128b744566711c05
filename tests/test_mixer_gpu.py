"""Whole mixer layers (hyena_mixer_*): projections, recurrence or FIR, projection and residual in a
row, forward, backward, token by token and captured, against the same layer in fp64 with autograd's
gradients (needs a B200).

Bounds, normwise (2-norm of the error over that of the value).  bf16: a value passes at most 8
roundings of half a step (2^-9 of the value in the mean square, 2^-8 at most) on its way, each
carried on by factors that leave its relative size about as it is: 8 x 2^-8 = 2^-5.  The FIR's
tensor path adds fp16 operands (2^-11), below that.  fp32: the products are within 2^-20 of sum
|x| |w|, the recurrence within 2^-18 of its terms at these lengths (the kernels' own tests), and
cancellation in sums over 96 to 300 terms takes up to 2^4 of it: 2^-13."""
import pytest
import torch

import gated_causal_fir_b200 as g

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
BOUND = {BF16: 2.0 ** -5, F32: 2.0 ** -13}


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from gated_causal_fir_b200 import build
    build.build()
    g.hyena_device_status(clear=True)
    yield
    assert g.hyena_device_status(clear=True) == 0, "a kernel raised its device status word"


def make(kind, E, D, d_g, dtype, seed=0, l_h=20):
    gen = torch.Generator().manual_seed(seed)

    def linear(n, k, shift=0.0):
        return g.Linear((torch.randn(n, k, generator=gen) / k ** 0.5).to(dtype).cuda(),
                        (0.3 * torch.randn(n, generator=gen) + shift).cuda())

    parts = dict(q=linear(D, E), k=linear(D, E), v=linear(D, E), out=linear(E, D), d_g=d_g)
    if kind == "scan":
        return g.MixerParams(gate=linear(D // d_g, E, 2.0), **parts)  # decays around 0.9
    return g.MixerParams(filters=(torch.randn(D // d_g, l_h, generator=gen) / l_h ** 0.5).cuda(),
                         **parts)


def reference(x, p, s0):
    """(out, state) in fp64 with grad, and the leaves."""
    leaves = {"x": x.double().requires_grad_()}
    for n in ("q", "k", "v", "out", "gate"):
        m = getattr(p, n)
        if m is not None:
            leaves[n + ".w"] = m.w.double().requires_grad_()
            leaves[n + ".b"] = m.b.double().requires_grad_()
    if p.filters is not None:
        leaves["filters"] = p.filters.double().requires_grad_()
    if s0 is not None:
        leaves["s0"] = s0.double().requires_grad_()
    lin = lambda n, t: t @ leaves[n + ".w"].t() + leaves[n + ".b"]  # noqa: E731
    xd = leaves["x"]
    q, k, v = lin("q", xd), lin("k", xd), lin("v", xd)
    L = x.shape[1]
    if p.gate is not None:
        a = torch.sigmoid(lin("gate", xd)).repeat_interleave(p.d_g, -1)
        s = leaves["s0"] if s0 is not None else torch.zeros_like(q[:, 0])
        ys = []
        for t in range(L):
            s = a[:, t] * s + k[:, t] * v[:, t]
            ys.append(q[:, t] * s)
        y, state = torch.stack(ys, 1), s
    else:
        h, kv, state = leaves["filters"].repeat_interleave(p.d_g, 0), k * v, None
        conv = sum(torch.nn.functional.pad(kv, (0, 0, j, 0))[:, :L] * h[:, j]
                   for j in range(min(L, h.shape[1])))
        y = q * conv
    return lin("out", y) + xd, state, leaves


def near(name, got, want, dtype):
    err = float((got.double() - want).norm() / want.norm())
    assert err <= BOUND[dtype], "%s: normwise error %.3g > %.3g" % (name, err, BOUND[dtype])


@pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "f32"))
@pytest.mark.parametrize("kind,B,L,E,D,d_g", (("scan", 2, 300, 128, 192, 64),
                                              ("scan", 1, 150, 96, 128, 1),
                                              ("scan", 3, 1, 64, 64, 8),
                                              ("scan", 1, 200, 100, 90, 6),
                                              ("fir", 2, 300, 128, 192, 64),
                                              ("fir", 1, 150, 96, 64, 16)))
def test_layer_forward_and_backward(kind, B, L, E, D, d_g, dtype):
    p = make(kind, E, D, d_g, dtype)
    gen = torch.Generator().manual_seed(9)
    x, dout = (torch.randn(B, L, E, generator=gen).to(dtype).cuda() for _ in range(2))
    s0 = ds = None
    if kind == "scan":
        s0, ds = (torch.randn(B, D, generator=gen).cuda() for _ in range(2))
    out, state, leaves = reference(x, p, s0)
    total = (out * dout.double()).sum()
    if ds is not None:
        total = total + (state * ds.double()).sum()
    names = list(leaves)
    want = dict(zip(names, torch.autograd.grad(total, [leaves[n] for n in names])))
    got, got_state, saved = g.hyena_mixer_fwd(x, p, s0=s0, save=True)
    near("out", got, out.detach(), dtype)
    dx, ds0, grads = g.hyena_mixer_bwd(x, p, saved, dout, ds_out=ds)
    near("dx", dx, want["x"], dtype)
    for n in ("q", "k", "v", "out", "gate"):
        if n + ".w" in want:
            near(n + ".w", grads[n][0], want[n + ".w"], dtype)
            near(n + ".b", grads[n][1], want[n + ".b"], dtype)
    if kind == "scan":
        near("state", got_state, state.detach(), dtype)
        near("ds0", ds0, want["s0"], dtype)
    else:
        near("filters", grads["filters"], want["filters"], dtype)
    again, _ = g.hyena_mixer_fwd(x, p, s0=s0)
    near("out without saving", again, out.detach(), dtype)


@pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "f32"))
def test_tokens_continue_a_prompt(dtype):
    """A prompt in one call and its next tokens one by one, eager and as a replayed graph, against
    the whole sequence."""
    B, L, E, D = 3, 40, 128, 192
    p = make("scan", E, D, 64, dtype, seed=4)
    x = torch.randn(B, L, E, generator=torch.Generator().manual_seed(2)).to(dtype).cuda()
    want, state, _ = reference(x, p, None)
    out, s = g.hyena_mixer_fwd(x[:, :32].contiguous(), p)
    near("prompt", out, want[:, :32].detach(), dtype)
    for t in range(32, 36):
        out, s = g.hyena_mixer_step(x[:, t].contiguous(), p, s)
        near("token %d" % t, out, want[:, t].detach(), dtype)
    tok = x[:, 36].contiguous()
    kept = s.clone()
    g.hyena_mixer_step(tok, p, kept.clone())  # everything loaded before the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = g.hyena_mixer_step(tok, p, s)
    s.copy_(kept)
    for t in range(36, L):
        tok.copy_(x[:, t])
        graph.replay()
        torch.cuda.synchronize()
        near("token %d" % t, out, want[:, t].detach(), dtype)
    near("state", s, state.detach(), dtype)


def test_captured_training_step():
    """Forward and backward of a layer in one graph, replayed on new inputs: the bits of the eager
    calls."""
    p = make("scan", 128, 128, 16, BF16, seed=7)
    x, dout = torch.randn(2, 200, 128, device="cuda").to(BF16), \
        torch.randn(2, 200, 128, device="cuda").to(BF16)

    def step():
        out, _, saved = g.hyena_mixer_fwd(x, p, save=True)
        dx, _, grads = g.hyena_mixer_bwd(x, p, saved, dout)
        return [out, dx] + [t for n in sorted(grads) for t in grads[n]]

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (1, 2):
        torch.manual_seed(seed)
        x.copy_(torch.randn(2, 200, 128))
        dout.copy_(torch.randn(2, 200, 128))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


def test_two_training_steps_at_once():
    """Two layers (time axis by clusters and by cuts) on two streams give what they give in turn."""
    jobs = []
    for L, E, D, d_g in ((2500, 128, 256, 64), (9000, 64, 64, 32)):
        p = make("scan", E, D, d_g, BF16)
        x, dout = (torch.randn(1, L, E, device="cuda").to(BF16) for _ in range(2))

        def step(p=p, x=x, dout=dout):
            out, state, saved = g.hyena_mixer_fwd(x, p, save=True)
            dx, ds0, grads = g.hyena_mixer_bwd(x, p, saved, dout)
            return [out, state, dx, ds0] + [t for n in sorted(grads) for t in grads[n]]
        jobs.append((step, step(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    results = [[], []]
    for _ in range(4):
        for i, (step, _, stream) in enumerate(jobs):
            with torch.cuda.stream(stream):
                results[i].append(step())
    torch.cuda.synchronize()
    for (_, alone, _), runs in zip(jobs, results):
        for run in runs:
            for a, b in zip(alone, run):
                assert torch.equal(a, b)


def test_refusals():
    p = make("fir", 64, 64, 16, BF16)
    x = torch.randn(1, 10, 64, device="cuda").to(BF16)
    with pytest.raises(ValueError):
        g.hyena_mixer_step(x[:, 0], p, torch.zeros(1, 64, device="cuda"))
    with pytest.raises(ValueError):
        g.hyena_mixer_fwd(x, p, s0=torch.zeros(1, 64, device="cuda"))
    saved = g.hyena_mixer_fwd(x, p, save=True)[2]
    with pytest.raises(ValueError):
        g.hyena_mixer_bwd(x, p, saved, x, ds_out=torch.zeros(1, 64, device="cuda"))
    with pytest.raises(ValueError):
        g.MixerParams(p.q, p.k, p.v, p.out, 16)
