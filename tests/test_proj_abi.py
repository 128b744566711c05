"""Host-side refusals and workspace sizes of the projections' C ABI (no GPU)."""
import pytest

import gated_causal_fir_b200 as g
from gated_causal_fir_b200 import _native, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _native.lib()


FWD = dict(x=1 << 24, w=2 << 24, bias=3 << 24, residual=4 << 24, y=5 << 24, z=6 << 24, M=64, N=128,
           K=72, act=1, dtype=0, ws=7 << 24, nws=1 << 24)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(w=None), 1), (dict(y=None), 1), (dict(M=-1), 1), (dict(N=0), 1),
    (dict(K=0), 1), (dict(act=-1), 1), (dict(act=5), 1), (dict(dtype=3), 1),
    (dict(M=1 << 31), 1), (dict(y=1 << 24), 1), (dict(y=2 << 24), 1), (dict(z=5 << 24), 1),
    (dict(z=4 << 24), 1), (dict(residual=(5 << 24) + 256), 1), (dict(bias=(5 << 24) + 64), 1),
    (dict(dtype=1, nws=1000), 1), (dict(dtype=1, ws=None), 1), (dict(dtype=1, ws=5 << 24), 1),
    (dict(x=(1 << 24) + 8), 3), (dict(y=(5 << 24) + 2), 3), (dict(bias=(3 << 24) + 2), 3),
    (dict(dtype=1, ws=(7 << 24) + 16), 3), (dict(M=0, x=None, y=None), 0),
])
def test_forward_refusals(lib, kw, code):
    a = dict(FWD, **kw)
    assert lib.hyena_proj_fwd(*[a[n] for n in FWD], None) == code


BWD = dict(x=1 << 24, w=2 << 24, z=3 << 24, dy=4 << 24, dx_add=5 << 24, dx=6 << 24, dw=7 << 24,
           db=8 << 24, M=64, N=128, K=72, act=1, dtype=0, ws=9 << 24, nws=1 << 24)


@pytest.mark.parametrize("kw,code", [
    (dict(dy=None), 1), (dict(z=None), 1), (dict(x=None), 1), (dict(w=None), 1),
    (dict(ws=None), 1), (dict(nws=64), 1), (dict(dx=1 << 24), 1), (dict(dw=6 << 24), 1),
    (dict(dx=(5 << 24) + 256), 1), (dict(dw=5 << 24), 1), (dict(db=(6 << 24) + 16), 1),
    (dict(act=7), 1), (dict(K=0), 1), (dict(ws=8 << 24), 1),
    (dict(dy=(4 << 24) + 4), 3), (dict(db=(8 << 24) + 1), 3), (dict(ws=(9 << 24) + 128), 3),
    (dict(M=0, dw=None, db=None), 0),
])
def test_backward_refusals(lib, kw, code):
    a = dict(BWD, **kw)
    assert lib.hyena_proj_bwd(*[a[n] for n in BWD], None) == code


def test_workspace_sizes(lib):
    assert g.hyena_proj_workspace_bytes(8192, 4096, 4096) == 0          # operands as they are
    assert g.hyena_proj_workspace_bytes(8192, 4096, 4095) > 0           # rows to be padded
    assert g.hyena_proj_workspace_bytes(100, 64, 64, g.HYENA_DTYPE_F32) >= 3 * 2 * 164 * 64
    assert g.hyena_proj_workspace_bytes(8, 256, 4096) == 0              # cut in a cluster
    assert g.hyena_proj_workspace_bytes(4096, 4096, 8192) > 0           # the last wave is cut
    assert g.hyena_proj_workspace_bytes(0, 8, 8) == 0
    assert g.hyena_proj_bwd_workspace_bytes(8192, 4096, 4096, "silu") >= 8192 * 4096 * 2
    with pytest.raises(g.HyenaError):
        g.hyena_proj_workspace_bytes(1, 0, 8)
