"""The fp64 reference of the gated linear recurrence against autograd and against differences
(host only), and the host-side refusals of the C ABI and of the Python entry points."""
import pytest
import torch

import gated_causal_fir_b200 as g
from gated_causal_fir_b200 import _native, build
from tests import _scan_ref as R


def _case(B, L, D, d_g, seed=0):
    gen = torch.Generator().manual_seed(seed)
    q, k, v, dy = (torch.randn(B, L, D, generator=gen, dtype=torch.float64) for _ in range(4))
    lg = -torch.rand(B, L, D // d_g, generator=gen, dtype=torch.float64)
    s0, ds = (torch.randn(B, D, generator=gen, dtype=torch.float64) for _ in range(2))
    return q, k, v, lg, s0, dy, ds


@pytest.mark.parametrize("d_g", (1, 2, 6))
def test_reference_gradients_are_autograds_and_differences(d_g):
    q, k, v, lg, s0, dy, ds = _case(2, 9, 6, d_g)
    leaves = [t.clone().requires_grad_() for t in (q, k, v, lg, s0)]

    def loss(q, k, v, lg, s0):
        s, total = s0, 0.0
        for t in range(q.shape[1]):
            s = lg[:, t].exp().repeat_interleave(d_g, -1) * s + k[:, t] * v[:, t]
            total = total + (dy[:, t] * q[:, t] * s).sum()
        return total + (ds * s).sum()

    auto = torch.autograd.grad(loss(*leaves), leaves)
    ref = R.Ref(q, k, v, lg, d_g, s0, dy, ds)
    for name, want in zip(("dq", "dk", "dv", "dg", "ds0"), auto):
        assert torch.allclose(ref.out[name][0], want, rtol=1e-12, atol=1e-12), name
    h, gen = 1e-6, torch.Generator().manual_seed(3)
    for i, name in enumerate(("dq", "dk", "dv", "dg", "ds0")):
        args = [q, k, v, lg, s0]
        way = torch.randn(args[i].shape, generator=gen, dtype=torch.float64)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + h * way, args[i] - h * way
        slope = float(loss(*up) - loss(*down)) / (2 * h)
        assert abs(slope - float((ref.out[name][0] * way).sum())) < 1e-6 * max(1, abs(slope)), name


def test_mixer_header_and_binding_agree():
    build.build()
    declared = _native.header_functions(_native.MIXER_HEADER_PATH)
    assert set(declared) == set(_native.MIXER_SIGNATURES)
    for name in declared:
        assert hasattr(_native.lib(), name), name


FWD = dict(q=1 << 20, k=2 << 20, v=3 << 20, g=4 << 20, s0=5 << 20, y=6 << 20, s_out=7 << 20,
           ckpt=8 << 20, B=2, L=300, D=64, d_g=16, dtype=0, ws=9 << 20, nws=1 << 20)


def _fwd(**kw):
    a = dict(FWD, **kw)
    return _native.lib().hyena_scan_fwd(*[a[n] for n in FWD], None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(g=None), 1), (dict(y=None), 1),
    (dict(B=-1), 1), (dict(L=-1), 1), (dict(D=0), 1), (dict(d_g=0), 1), (dict(d_g=48), 1),
    (dict(dtype=2), 1), (dict(B=1 << 40, L=1 << 20), 1), (dict(L=1 << 31), 1),
    (dict(y=(1 << 20) + 64), 1), (dict(s_out=5 << 20), 1), (dict(ckpt=6 << 20), 1),
    (dict(s_out=(6 << 20) + 128), 1), (dict(ws=None), 1), (dict(nws=256), 1),
    (dict(q=(1 << 20) + 1), 3), (dict(s0=(5 << 20) + 2), 3), (dict(ws=(9 << 20) + 8), 3),
    (dict(dtype=1, v=(3 << 20) + 2), 3), (dict(B=0), 0),
])
def test_forward_refusals(kw, code):
    build.build()
    # a long narrow problem needs a workspace; the others here do not
    base = dict(L=100000, D=64, B=1) if "ws" in kw or "nws" in kw else {}
    far = {n: (i + 1) << 32 for i, n in enumerate(("q", "k", "v", "g", "s0", "y", "s_out", "ckpt"))}
    assert _fwd(**dict(dict(base, **far) if base else {}, **kw)) == code


BWD = dict(q=1 << 20, k=2 << 20, v=3 << 20, g=4 << 20, s0=5 << 20, dy=6 << 20, ds_out=7 << 20,
           ckpt=8 << 20, dq=9 << 20, dk=10 << 20, dv=11 << 20, dg=12 << 20, ds0=13 << 20, B=2,
           L=300, D=64, d_g=64, dtype=0, ws=14 << 20, nws=1 << 20)


@pytest.mark.parametrize("kw,code", [
    (dict(dy=None), 1), (dict(dq=None), 1), (dict(dk=None), 1), (dict(dv=None), 1),
    (dict(dg=None), 1), (dict(dq=10 << 20), 1), (dict(dk=1 << 20), 1), (dict(ds0=7 << 20), 1),
    (dict(dg=8 << 20), 1), (dict(ws=None), 1), (dict(nws=0), 1), (dict(ws=9 << 20), 1),
    (dict(dg=(12 << 20) + 1), 3), (dict(ds0=(13 << 20) + 2), 3), (dict(D=63), 1), (dict(B=0), 0),
])
def test_backward_refusals(kw, code):
    build.build()
    a = dict(BWD, **kw)
    assert _native.lib().hyena_scan_bwd(*[a[n] for n in BWD], None) == code


STEP = dict(q=1 << 20, k=2 << 20, v=3 << 20, g=4 << 20, s=5 << 20, y=6 << 20, s_out=7 << 20, B=2,
            D=64, d_g=16, dtype=0)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(s=None), 1), (dict(s_out=None), 1), (dict(y=5 << 20), 1),
    (dict(s_out=(5 << 20) + 256), 1), (dict(y=1 << 20), 1), (dict(d_g=5), 1), (dict(dtype=9), 1),
    (dict(k=(2 << 20) + 1), 3), (dict(s=(5 << 20) + 2), 3), (dict(B=0), 0),
])
def test_step_refusals(kw, code):
    build.build()
    a = dict(STEP, **kw)
    assert _native.lib().hyena_scan_step(*[a[n] for n in STEP], None) == code


def test_sizes_of_workspaces_and_checkpoints():
    build.build()
    lib = _native.lib()
    assert lib.hyena_scan_ckpt_tiles(0, 0) == 0 and lib.hyena_scan_ckpt_tiles(1, 0) == 1
    assert lib.hyena_scan_ckpt_tiles(-1, 0) == -1 and lib.hyena_scan_ckpt_tiles(1, 5) == -1
    assert g.hyena_scan_workspace_bytes(1, 8192, 4096, 64) == 0     # enough channels
    assert g.hyena_scan_workspace_bytes(1, 65536, 64, 16) > 0       # cut along time
    assert g.hyena_scan_workspace_bytes(1, 100, 64, 16) == 0        # too short to cut
    full = g.hyena_scan_bwd_workspace_bytes(1, 8192, 4096, 64)
    assert full >= 8192 * 128 * 4                                   # one dg partial per 32 channels
    assert g.hyena_scan_bwd_workspace_bytes(1, 8192, 4096, 64, have_ckpt=False) > full
    assert g.hyena_scan_bwd_workspace_bytes(1, 8192, 4096, 16) == 0
    with pytest.raises(g.HyenaError):
        g.hyena_scan_workspace_bytes(1, 8, 7, 2)


def test_python_entry_points_refuse_host_tensors():
    t = torch.zeros(1, 4, 8)
    with pytest.raises(TypeError):
        g.hyena_scan_fwd(t, t, t, t, 1)
    with pytest.raises(TypeError):
        g.hyena_scan_step(t[:, 0], t[:, 0], t[:, 0], t[:, 0], t[:, 0], 1)
