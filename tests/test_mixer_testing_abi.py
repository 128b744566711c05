"""Host-side refusals of the mixer operators' test entry points, and of sizes (no GPU)."""
import pytest

from gated_causal_fir_b200 import _native, build

ARGS = dict(x=1 << 24, w=2 << 24, residual=3 << 24, y=4 << 24, M=64, N=128, K=72, fault=0,
            wait_ns=20_000_000)


@pytest.mark.parametrize("kw,code", [
    (dict(fault=-1), 1), (dict(fault=9), 1), (dict(wait_ns=1000), 1), (dict(wait_ns=3 * 10**9), 1),
    (dict(N=100), 2), (dict(K=60), 2), (dict(M=4096, N=4096, K=8192, y=1 << 40), 2), (dict(x=None), 1), (dict(y=1 << 24), 1),
    (dict(x=(1 << 24) + 2), 3), (dict(M=0), 0)])
def test_refusals(kw, code):
    build.build()
    a = dict(ARGS, **kw)
    assert _native.lib().hyena_testing_proj_fault(*[a[n] for n in ARGS], None) == code


BIG = 1 << 30


@pytest.mark.parametrize("M,N,K", ((BIG, BIG, 8), (BIG, BIG, 1 << 24), (1 << 26, 1 << 26, 1 << 20)))
def test_more_tiles_than_can_be_counted_are_refused(M, N, K):
    """By the size queries as by the calls, for the product itself and as a backward's."""
    build.build()
    lib = _native.lib()
    assert lib.hyena_proj_workspace_bytes(M, N, K, 0) == -2
    at = [(i + 1) << 58 for i in range(4)]
    assert lib.hyena_proj_fwd(at[0], at[1], None, None, at[2], None, M, N, K, 0, 0, None, 0,
                              None) == 2
    m = min(M, 8388480)
    assert lib.hyena_proj_bwd_workspace_bytes(m, 1 << 24, 1 << 24, 0, 0) == -2
    assert lib.hyena_proj_bwd_workspace_bytes(8388481, 8, 8, 0, 0) == -2
    assert lib.hyena_proj_bwd_workspace_bytes(8, (1 << 24) + 1, 8, 0, 0) == -2
    assert lib.hyena_proj_bwd_workspace_bytes(8388480, 8, 8, 0, 0) > 0


SCAN = dict(q=1 << 24, k=2 << 24, v=3 << 24, g=4 << 24, y=5 << 24, s_out=6 << 24, B=1, L=1250, D=320,
            d_g=64, dtype=0, fault=0, wait_ns=20_000_000)


@pytest.mark.parametrize("kw,code", [
    (dict(fault=2), 1), (dict(fault=-1), 1), (dict(wait_ns=10), 1), (dict(wait_ns=1 << 40), 1),
    (dict(L=100), 2), (dict(D=4096), 2), (dict(q=None), 1), (dict(d_g=7), 1), (dict(y=1 << 24), 1)])
def test_scan_refusals(kw, code):
    build.build()
    a = dict(SCAN, **kw)
    assert _native.lib().hyena_testing_scan_fault(*[a[n] for n in SCAN], None) == code
