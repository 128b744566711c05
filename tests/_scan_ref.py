"""The gated linear recurrence in fp64 on the CPU, straight from its definition, with the bounds
its fp32 evaluation must keep.

Bounds.  Let u = 2^-24.  One token of the recurrence costs, relative to the terms it adds up:
expf at most 2 ulp (4 u), x = k v (u), the fused multiply-add (u), and where runs of tokens are
joined a rounding of the run's decay product and of its join (2 u): at most 8 u, of terms whose
sizes add up to m_t = a_t m_{t-1} + |x_t|.  An error once made decays like the state.  So the error
of s_t is at most e_t = a_t e_{t-1} + 8 u m_t, to first order in u; ``SLACK`` = 2 covers the
second order and the roundings of m and e themselves.  The gradients obey the same recurrence
backwards in time, and a product of two such values has the sum of their relative errors plus u.
A result is then rounded once: half a step of its type, 2^-8 (bf16) or 2^-24 (fp32) of its size.
"""
import torch

U = 2.0 ** -24
SLACK = 2.0
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _wide(t, d_g):
    return t.repeat_interleave(d_g, -1)


def _sum(t, d_g):
    return t.reshape(*t.shape[:-1], -1, d_g).sum(-1)


def recur(a, x, s0):
    """[B, L, D] states s_t = a_t s_{t-1} + x_t from s0 [B, D]."""
    out, s = torch.empty_like(x), s0
    for t in range(x.shape[1]):
        s = a[:, t] * s + x[:, t]
        out[:, t] = s
    return out


def _back(a, z, w):
    """u_t = z_t + a_{t+1} u_{t+1}, w reaching the last; also a_0 u_0."""
    out = torch.empty_like(z)
    for t in range(z.shape[1] - 1, -1, -1):
        out[:, t] = z[:, t] + w
        w = a[:, t] * out[:, t]
    return out, w


class Ref:
    """Results and bounds of the forward, and with dy of the backward, as {name: (value, error
    bound before the final rounding)}."""

    def __init__(self, q, k, v, g, d_g, s0=None, dy=None, ds_out=None):
        d = [t.detach().cpu().double() if t is not None else None
             for t in (q, k, v, g, s0, dy, ds_out)]
        q, k, v, g, s0, dy, ds_out = d
        B, L, D = q.shape
        zero = torch.zeros(B, D, dtype=torch.float64)
        s0 = zero if s0 is None else s0
        a, x = _wide(torch.exp(g), d_g), k * v
        s = recur(a, x, s0)
        m = recur(a, x.abs(), s0.abs())
        e = SLACK * recur(a, 8 * U * m, zero)
        last = (s[:, -1], e[:, -1]) if L else (s0, zero)
        self.out = {"y": (q * s, q.abs() * e + U * (q * s).abs()), "s_out": last}
        if dy is None:
            return
        ds_out = zero if ds_out is None else ds_out
        z = q * dy
        ut, w0 = _back(a, z, ds_out)
        mu, _ = _back(a, z.abs(), ds_out.abs())
        eu, ew = _back(a, 8 * U * mu, zero)
        eu, ew = SLACK * eu, SLACK * ew
        before = torch.cat((s0[:, None], s[:, :-1]), 1)
        eb = torch.cat((zero[:, None], e[:, :-1]), 1)
        dg = a * before * ut
        edg = a * (before.abs() * eu + ut.abs() * eb + eb * eu) + 8 * U * dg.abs()
        # the group's sum: at most d_g roundings of partial sums no larger than the terms' sizes
        edg = _sum(edg, d_g) + d_g * U * _sum(dg.abs(), d_g)
        self.out.update(
            dq=(dy * s, dy.abs() * e + U * (dy * s).abs()),
            dk=(ut * v, v.abs() * eu + U * (ut * v).abs()),
            dv=(ut * k, k.abs() * eu + U * (ut * k).abs()),
            dg=(_sum(dg, d_g), edg), ds0=(w0, ew + 8 * U * w0.abs()))


def check(name, got, ref):
    """``got`` within the bound of ref.out[name] and its type's final rounding."""
    want, err = ref.out[name]
    got_d = got.detach().cpu().double()
    assert got_d.shape == want.shape, (name, got_d.shape, want.shape)
    tol = err * (1 + HALF_STEP[got.dtype]) + HALF_STEP[got.dtype] * want.abs() + 1e-37
    bad = ~((got_d - want).abs() <= tol)
    assert not bad.any(), "%s: %d of %d values out of bounds, worst error/bound %.3g, first at %s" % (
        name, int(bad.sum()), bad.numel(),
        float(((got_d - want).abs() / tol)[bad].max()), bad.nonzero()[0].tolist())
