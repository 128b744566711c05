"""The gated linear recurrence (C: ``hyena_scan_*`` of ``include/hyena_mixer.h``).

    x_t = k_t v_t,   s_t = exp(g_t) s_{t-1} + x_t,   y_t = q_t s_t

over [B, L, D] tensors, with one log decay g <= 0 for each token and group of d_g channels: the
gates of the FIR operator around a state that the data lets decay.  The functions marshal torch
CUDA tensors into pointers, sizes and a stream; outputs and workspaces that are not given come
from torch.
"""
from ._args import (CODES, code as code_of, cuda_tensor, like, made, nbytes, need, ptr, run,
                    stream_handle, torch_, workspace as workspace_of)
from ._native import HYENA_DTYPE_BF16


def _shapes(q, k, v, g, d_g, dims):
    """The type code of q [*dims, D], k, v like it and g [*dims, D // d_g]."""
    try:  # the calls that are right, quickly
        shape, dtype, device = q.shape, q.dtype, q.device
        code = CODES.get(dtype)
        if (code is not None and q.is_cuda and len(shape) == len(dims) // 3 + 1
                and shape[-1] % d_g == 0 and q.is_contiguous()
                and like(k, shape, dtype, device) and like(v, shape, dtype, device)
                and like(g, shape if d_g == 1 else shape[:-1] + (shape[-1] // d_g,), dtype,
                         device) and type(d_g) is int and d_g > 0 and shape[-1] > 0):
            return code
    except (AttributeError, TypeError, ZeroDivisionError):
        pass
    cuda_tensor("q", q, "[%s] tensor" % dims)
    shape, dtype, device = q.shape, q.dtype, q.device
    if len(shape) != len(dims) // 3 + 1:
        raise TypeError("q must be a CUDA [%s] tensor" % dims)
    code = code_of(q, "q")
    D = shape[-1]
    if not isinstance(d_g, int) or d_g < 1 or D < 1 or D % d_g != 0:
        raise ValueError("d_g = %s must divide D = %d" % (d_g, D))
    need("q", q, shape, dtype, device)
    need("k", k, shape, dtype, device)
    need("v", v, shape, dtype, device)
    need("g", g, shape if d_g == 1 else shape[:-1] + (D // d_g,), dtype, device)
    return code


def _state(name, t, q):
    if t is not None:
        need(name, t, (q.shape[0], q.shape[-1]), torch_().float32, q.device)


def hyena_scan_workspace_bytes(B, L, D, d_g, dtype=HYENA_DTYPE_BF16):
    """Host-only: device workspace bytes hyena_scan_fwd needs for this shape."""
    return nbytes("hyena_scan_workspace_bytes", B, L, D, d_g, dtype)


def hyena_scan_bwd_workspace_bytes(B, L, D, d_g, dtype=HYENA_DTYPE_BF16, have_ckpt=True):
    """Host-only: device workspace bytes hyena_scan_bwd needs for this shape."""
    return nbytes("hyena_scan_bwd_workspace_bytes", B, L, D, d_g, dtype, 1 if have_ckpt else 0)


def hyena_scan_ckpt(q):
    """An uninitialised checkpoint tensor for sequences like q [B, L, D]: fp32 [B, tiles, D]."""
    torch = torch_()
    tiles = nbytes("hyena_scan_ckpt_tiles", q.shape[1], code_of(q, "q"))
    return torch.empty((q.shape[0], tiles, q.shape[2]), dtype=torch.float32, device=q.device)


def _ckpt(t, q, code):
    if t is None:
        return None
    tiles = nbytes("hyena_scan_ckpt_tiles", q.shape[1], code)
    return need("ckpt", t, (q.shape[0], tiles, q.shape[2]), torch_().float32, q.device)


def hyena_scan_fwd(q, k, v, g, d_g, s0=None, y=None, s_out=None, ckpt=None, workspace=None,
                   stream=None):
    """Forward; returns (y, s_out).

    q, k, v: CUDA [B, L, D], all bf16 or all fp32.  g: [B, L, D // d_g] of the same type, log
    decays <= 0; -inf drops the state before its token.  s0: fp32 [B, D], the state before the
    first token (zeros when None).  s_out: fp32 [B, D], the state after the last.  ckpt: a
    tensor of hyena_scan_ckpt(q), filled for hyena_scan_bwd.  Runs asynchronously on ``stream``
    (default: the current stream of q's device), which waits for nothing queued on others.
    """
    code = _shapes(q, k, v, g, d_g, "B, L, D")
    B, L, D = q.shape
    device = q.device
    _state("s0", s0, q)
    _ckpt(ckpt, q, code)
    if y is None:
        y = made(stream, q.device, lambda: torch_().empty_like(q))
    else:
        need("y", y, q.shape, q.dtype, device)
    if s_out is None:
        s_out = made(stream, device, lambda: torch_().empty_like(s0) if s0 is not None else
                     torch_().empty((B, D), dtype=torch_().float32, device=device))
    else:
        _state("s_out", s_out, q)
    size = nbytes("hyena_scan_workspace_bytes", B, L, D, d_g, code)
    ws, nws, _buf = workspace_of(workspace, size, device, stream)
    run("hyena_scan_fwd", device, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), ptr(s0),
        y.data_ptr(), s_out.data_ptr(), ptr(ckpt), B, L, D, d_g, code, ws, nws,
        stream_handle(device, stream))
    return y, s_out


def hyena_scan_bwd(q, k, v, g, dy, d_g, s0=None, ds_out=None, ckpt=None, grads=None,
                   workspace=None, stream=None):
    """Gradients (dq, dk, dv, dg, ds0) of hyena_scan_fwd for dy (of y) and ds_out (of the last
    state; fp32 [B, D], zeros when None).

    ckpt: as hyena_scan_fwd filled it for the same inputs; without it a pass over k, v and g
    finds the states again.  grads: optional preallocated (dq, dk, dv, dg, ds0), overwritten.
    """
    torch = torch_()
    code = _shapes(q, k, v, g, d_g, "B, L, D")
    B, L, D = q.shape
    need("dy", dy, q.shape, q.dtype, q.device)
    _state("s0", s0, q)
    _state("ds_out", ds_out, q)
    _ckpt(ckpt, q, code)
    given = grads is not None
    if not given:
        grads = [made(stream, q.device, lambda t=t: torch.empty_like(t)) for t in (q, q, q, g)]
        grads.append(made(stream, q.device,
                          lambda: torch.empty((B, D), dtype=torch.float32, device=q.device)))
    dq, dk, dv, dg, ds0 = grads
    if given:
        for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
            need(name, t, q.shape, q.dtype, q.device)
        need("dg", dg, g.shape, g.dtype, q.device)
        if ds0 is None:
            raise ValueError("ds0 must be an fp32 [B, D] tensor")
        _state("ds0", ds0, q)
    size = nbytes("hyena_scan_bwd_workspace_bytes", B, L, D, d_g, code, int(ckpt is not None))
    ws, nws, _buf = workspace_of(workspace, size, q.device, stream)
    run("hyena_scan_bwd", q.device, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(),
        ptr(s0), dy.data_ptr(), ptr(ds_out), ptr(ckpt), dq.data_ptr(), dk.data_ptr(),
        dv.data_ptr(), dg.data_ptr(), ds0.data_ptr(), B, L, D, d_g, code, ws, nws,
        stream_handle(q.device, stream))
    return dq, dk, dv, dg, ds0


def hyena_scan_step(q, k, v, g, state, d_g, y=None, state_out=None, stream=None):
    """One token of B running sequences; returns (y, state_out).

    q, k, v: CUDA [B, D]; g: [B, D // d_g]; state: fp32 [B, D].  state_out None advances
    ``state`` in place."""
    code = _shapes(q, k, v, g, d_g, "B, D")
    B, D = q.shape
    if state is None:
        raise ValueError("state must be an fp32 [B, D] tensor")
    _state("state", state, q)
    if state_out is None:
        state_out = state
    else:
        _state("state_out", state_out, q)
    if y is None:
        y = made(stream, q.device, lambda: torch_().empty_like(q))
    else:
        need("y", y, q.shape, q.dtype, q.device)
    run("hyena_scan_step", q.device, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(),
        state.data_ptr(), y.data_ptr(), state_out.data_ptr(), B, D, d_g, code,
        stream_handle(q.device, stream))
    return y, state_out
