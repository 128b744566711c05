"""A mixer layer: projections, a gated sequence mixer, and the projection back into the residual
stream.

    q, k, v = x w_q^T + b_q, ...        y = mixer(q, k, v)        out = x + y w_o^T + b_o

The mixer is the gated causal FIR of this package (``filters`` given: the Hyena-SE / Hyena-MR
operator, whose q, k and v are projections of the layer's input, StripedHyena 2 overview page,
Sec. 3) or the gated linear recurrence with decays from a fourth projection (``gate`` given),

    g = log sigmoid(x w_g^T + b_g),

one for each group of d_g channels.  Forward, backward and, for the recurrence, one token of
running sequences; every product, scan and convolution is a kernel of this package.  x: CUDA
[B, L, E], bf16 or fp32, weights of the same type, biases fp32.
"""
from dataclasses import dataclass
from typing import Any, Optional

from ._args import torch_
from .projection import hyena_proj_bwd, hyena_proj_fwd
from .recurrence import hyena_scan_bwd, hyena_scan_ckpt, hyena_scan_fwd, hyena_scan_step


@dataclass
class Linear:
    """w [N, K] with an optional fp32 bias [N]."""
    w: Any
    b: Any = None


@dataclass
class MixerParams:
    """q, k, v: Linear [D, E]; out: Linear [E, D]; either ``gate``, Linear [D // d_g, E], for the
    recurrence, or ``filters``, fp32 [D // d_g, l_h], for the FIR (block size l_b)."""
    q: Linear
    k: Linear
    v: Linear
    out: Linear
    d_g: int
    gate: Optional[Linear] = None
    filters: Any = None
    l_b: int = 64

    def __post_init__(self):
        if (self.gate is None) == (self.filters is None):
            raise ValueError("a mixer has a gate (recurrence) or filters (FIR)")


def _fir(p, q, k, v):
    import gated_causal_fir_b200 as fir
    bf16 = q.dtype == torch_().bfloat16
    return (fir.hyena_conv_fwd if bf16 else fir.hyena_conv_fwd_f32)(q, k, v, p.filters, p.d_g,
                                                                    p.l_b)


def hyena_mixer_fwd(x, p, s0=None, save=False):
    """(out, state) or, with ``save``, (out, state, saved) for hyena_mixer_bwd.

    s0, state: fp32 [B, D], the recurrence's state before the first and after the last token (None
    for the FIR).  Runs on the current stream."""
    q, k, v = (hyena_proj_fwd(x, m.w, m.b) for m in (p.q, p.k, p.v))
    g = z = ckpt = state = None
    if p.gate is not None:
        z = x.new_empty(x.shape[:-1] + (p.gate.w.shape[0],)) if save else None
        g = hyena_proj_fwd(x, p.gate.w, p.gate.b, act="logsigmoid", z=z)
        ckpt = hyena_scan_ckpt(q) if save else None
        y, state = hyena_scan_fwd(q, k, v, g, p.d_g, s0=s0, ckpt=ckpt)
    else:
        if s0 is not None:
            raise ValueError("the FIR keeps no state")
        y = _fir(p, q, k, v)
    out = hyena_proj_fwd(y, p.out.w, p.out.b, residual=x)
    return (out, state, (q, k, v, g, z, ckpt, y, s0)) if save else (out, state)


def hyena_mixer_bwd(x, p, saved, dout, ds_out=None):
    """(dx, ds0, grads) for dout (of out) and ds_out (of the last state): grads maps "q", "k", "v",
    "out" and "gate" to (dw, db) and "filters" to its gradient.

    dx is added up by the projections' products, the first onto the residual branch's gradient and
    the others in place: without passes of its own, at the price of a rounding to x's type for each
    of the three or four (for bf16, half a step of the sum so far each time)."""
    import gated_causal_fir_b200 as fir
    if ds_out is not None and p.gate is None:
        raise ValueError("the FIR keeps no state")
    q, k, v, g, z, ckpt, y, s0 = saved
    grads = {}
    dy, *grads["out"] = hyena_proj_bwd(y, p.out.w, dout)
    ds0 = None
    if p.gate is not None:
        dq, dk, dv, dg, ds0 = hyena_scan_bwd(q, k, v, g, dy, p.d_g, s0=s0, ds_out=ds_out,
                                             ckpt=ckpt)
        dx, *grads["gate"] = hyena_proj_bwd(x, p.gate.w, dg, z=z, act="logsigmoid", dx_add=dout)
        so_far = dx
    else:
        dq, dk, dv, grads["filters"] = fir.hyena_conv_bwd(q, k, v, p.filters, dy, p.d_g, p.l_b)
        dx, so_far = torch_().empty_like(x), dout
    for name, m, d in (("q", p.q, dq), ("k", p.k, dk), ("v", p.v, dv)):
        dw, db = torch_().empty_like(m.w), m.w.new_empty((m.w.shape[0],), dtype=torch_().float32)
        hyena_proj_bwd(x, m.w, d, dx_add=so_far, grads=(dx, dw, db))
        grads[name], so_far = [dw, db], dx
    return dx, ds0, {n: tuple(d) if isinstance(d, list) else d for n, d in grads.items()}


def hyena_mixer_step(x, p, state):
    """One token x [B, E] of B running sequences: (out, state), the state advanced in place."""
    if p.gate is None:
        raise ValueError("single tokens need the recurrence; the FIR continues a sequence by "
                         "hyena_conv_fwd_hist")
    q, k, v = (hyena_proj_fwd(x, m.w, m.b) for m in (p.q, p.k, p.v))
    g = hyena_proj_fwd(x, p.gate.w, p.gate.b, act="logsigmoid")
    y, state = hyena_scan_step(q, k, v, g, state, p.d_g)
    return hyena_proj_fwd(y, p.out.w, p.out.b, residual=x), state
