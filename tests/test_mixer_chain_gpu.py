"""Chains of the package's kernels without waits between them, where each lets the next one start
before it has finished: what a later kernel reads is what the earlier ones wrote in this pass (needs
a B200).  The inputs change from pass to pass in the same buffers, so that a value read too early is
the last pass's."""
import pytest
import torch

import gated_causal_fir_b200 as g
from tests.test_mixer_gpu import make

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


class Layer:
    """A FIR mixer layer's forward and backward, by calls into buffers of its own; `pause` runs
    between any two calls."""

    def __init__(self, B, L, E, D, d_g, l_h, dtype):
        self.p = make("fir", E, D, d_g, dtype, l_h=l_h)
        new = lambda *s, dt=dtype: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
        self.x, self.dout, self.out = (new(B, L, E) for _ in range(3))
        self.q, self.k, self.v, self.y, self.dy = (new(B, L, D) for _ in range(5))
        self.gy = (self.dy, new(E, D), new(E, dt=F32))
        self.gf = [new(B, L, D) for _ in range(3)] + [torch.zeros_like(self.p.filters)]
        self.dx = new(B, L, E)
        self.gp = [(self.dx, new(D, E), new(D, dt=F32)) for _ in range(3)]
        self.ws = new(g.hyena_conv_bwd_workspace_bytes(B, L, D, d_g, l_h) + 256, dt=torch.uint8)

    def outputs(self):
        return [self.out, self.y, *self.gy, *self.gf, self.dx] + [t for gp in self.gp for t in gp]

    def run(self, pause=lambda: None):
        p, n = self.p, self.p.d_g
        for m, o in ((p.q, self.q), (p.k, self.k), (p.v, self.v)):
            g.hyena_proj_fwd(self.x, m.w, m.b, y=o)
            pause()
        g.hyena_conv_fwd_ex(self.q, self.k, self.v, p.filters, n, 64, y=self.y)
        pause()
        g.hyena_proj_fwd(self.y, p.out.w, p.out.b, residual=self.x, y=self.out)
        pause()
        g.hyena_proj_bwd(self.y, p.out.w, self.dout, grads=self.gy)
        pause()
        g.hyena_conv_bwd(self.q, self.k, self.v, p.filters, self.dy, n, 64, grads=self.gf,
                         workspace=self.ws)
        pause()
        add = self.dout
        for m, d, gp in zip((p.q, p.k, p.v), self.gf, self.gp):
            g.hyena_proj_bwd(self.x, m.w, d, dx_add=add, grads=gp)
            add = self.dx
            pause()


# the FIR's kernels by l_h, d_g and type: tensor cores (forward and backward), register window,
# tiled direct sums, the block FFT; small and ordinary sizes
LAYERS = [(1, 64, 64, 64, 64, 20, BF16), (1, 300, 128, 192, 64, 7, BF16),
          (2, 1500, 256, 512, 64, 128, BF16), (1, 700, 128, 128, 16, 7, BF16),
          (1, 2000, 256, 1024, 16, 13, BF16), (2, 300, 64, 96, 16, 7, F32),
          (1, 500, 64, 66, 6, 30, BF16), (1, 3000, 64, 128, 64, 700, BF16),
          (1, 1200, 64, 64, 64, 300, F32)]


@pytest.mark.parametrize("layer", LAYERS, ids=["x".join(map(str, s[:6])) + str(s[6])[-4:]
                                               for s in LAYERS])
def test_a_training_step_reads_what_this_pass_wrote(layer):
    B, L, E, D = layer[:4]
    chain = Layer(*layer)
    inputs = [[torch.randn(B, L, E, device="cuda").to(layer[6]) for _ in range(2)]
              for _ in range(3)]
    want = []
    for x, dout in inputs:
        chain.x.copy_(x)
        chain.dout.copy_(dout)
        chain.run(torch.cuda.synchronize)
        want.append([t.clone() for t in chain.outputs()])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        chain.run()
    for i in range(12):
        for run in (chain.run, graph.replay):
            chain.x.copy_(inputs[i % 3][0])
            chain.dout.copy_(inputs[i % 3][1])
            run()
            for a, b in zip(chain.outputs(), want[i % 3]):
                assert torch.equal(a, b)


@pytest.mark.parametrize("layer", LAYERS[:6], ids=["x".join(map(str, s[:6])) + str(s[6])[-4:]
                                                   for s in LAYERS[:6]])
def test_the_layers_backward_is_the_chain_of_its_calls(layer):
    """The same bits as the calls one by one, and what comes in stays as it was."""
    chain = Layer(*layer)
    chain.x.copy_(torch.randn_like(chain.x))
    chain.dout.copy_(torch.randn_like(chain.dout))
    chain.run(torch.cuda.synchronize)
    kept = chain.x.clone(), chain.dout.clone()
    out, _, saved = g.hyena_mixer_fwd(chain.x, chain.p, save=True)
    dx, ds0, grads = g.hyena_mixer_bwd(chain.x, chain.p, saved, chain.dout)
    assert torch.equal(out, chain.out) and torch.equal(dx, chain.dx) and ds0 is None
    assert dx.data_ptr() != chain.dout.data_ptr()
    for n, gp in zip("qkv", chain.gp):
        assert torch.equal(grads[n][0], gp[1]) and torch.equal(grads[n][1], gp[2])
    assert torch.equal(grads["out"][0], chain.gy[1]) and torch.equal(grads["filters"], chain.gf[3])
    assert torch.equal(chain.x, kept[0]) and torch.equal(chain.dout, kept[1])
