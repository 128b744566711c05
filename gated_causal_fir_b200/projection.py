"""The projections around a sequence mixer (C: ``hyena_proj_*`` of ``include/hyena_mixer.h``).

    y = act(x w^T + bias) + residual        act: none, gelu, silu, sigmoid, logsigmoid

x: CUDA [..., K], w: [N, K], all bf16 or all fp32; bias fp32 [N].  The functions marshal torch
CUDA tensors into pointers, sizes and a stream; outputs and workspaces that are not given come
from torch.
"""
from ._args import (CODES, code as code_of, cuda_tensor, made, nbytes, need, ptr, run,
                    stream_handle, torch_, workspace as workspace_of)
from ._native import ACT_CODES, HYENA_DTYPE_BF16


def _act(act):
    try:
        return ACT_CODES[act]
    except (KeyError, TypeError):
        raise ValueError("act must be one of %s, got %r" % (", ".join(ACT_CODES), act)) from None


def _rows(x, w):
    """(type code, M, N, K) of x [..., K] and w [N, K]."""
    try:  # the calls that are right, quickly
        shape, dtype, device = x.shape, x.dtype, x.device
        code, (N, K) = CODES.get(dtype), w.shape
        if (code is not None and x.is_cuda and len(shape) > 1 and shape[-1] == K and N > 0 and K > 0
                and w.dtype is dtype and w.device == device and x.is_contiguous()
                and w.is_contiguous()):
            return code, x.numel() // K, N, K
    except (AttributeError, TypeError, ValueError):
        pass
    cuda_tensor("x", x, "[..., K] tensor")
    shape = x.shape
    if len(shape) < 2:
        raise TypeError("x must be a CUDA [..., K] tensor of at least two dimensions")
    code = code_of(x, "x")
    K = shape[-1]
    need("x", x, shape, x.dtype, x.device)
    cuda_tensor("w", w, "[N, K] tensor")
    N = w.shape[0]
    if N < 1 or K < 1:
        raise ValueError("w must not be empty")
    need("w", w, (N, K), x.dtype, x.device)
    return code, x.numel() // K, N, K


def hyena_proj_workspace_bytes(M, N, K, dtype=HYENA_DTYPE_BF16):
    """Host-only: device workspace bytes hyena_proj_fwd needs for this shape."""
    return nbytes("hyena_proj_workspace_bytes", M, N, K, dtype)


def hyena_proj_bwd_workspace_bytes(M, N, K, act="none", dtype=HYENA_DTYPE_BF16):
    """Host-only: device workspace bytes hyena_proj_bwd needs for this shape."""
    return nbytes("hyena_proj_bwd_workspace_bytes", M, N, K, _act(act), dtype)


def hyena_proj_fwd(x, w, bias=None, act="none", residual=None, y=None, z=None, workspace=None,
                   stream=None):
    """y = act(x w^T + bias) + residual, [..., N]; returns y.

    z: optional [..., N] tensor of x's type that receives the value before the activation, for
    hyena_proj_bwd.  y may be ``residual`` itself.  Tensors start on 16-byte boundaries (views into
    others may not), biases on 4-byte ones.  Runs asynchronously on ``stream`` (default: the
    current stream of x's device), which waits for nothing queued on others.
    """
    act = _act(act)
    code, M, N, K = _rows(x, w)
    shape = x.shape[:-1] + (N,)
    if bias is not None:
        need("bias", bias, (N,), torch_().float32, x.device)
    if residual is not None:
        need("residual", residual, shape, x.dtype, x.device)
    if z is not None:
        need("z", z, shape, x.dtype, x.device)
    if y is None:
        y = made(stream, x.device, lambda: x.new_empty(shape) if residual is None else
                 torch_().empty_like(residual))
    else:
        need("y", y, shape, x.dtype, x.device)
    size = nbytes("hyena_proj_workspace_bytes", M, N, K, code)
    ws, nws, _buf = workspace_of(workspace, size, x.device, stream)
    run("hyena_proj_fwd", x.device, x.data_ptr(), w.data_ptr(), ptr(bias), ptr(residual),
        y.data_ptr(), ptr(z), M, N, K, act, code, ws, nws, stream_handle(x.device, stream))
    return y


def hyena_proj_bwd(x, w, dy, z=None, act="none", dx_add=None, grads=None, workspace=None,
                   stream=None):
    """Gradients (dx, dw, db) of hyena_proj_fwd for dy [..., N]; the residual's is dy itself.

    z: as the forward left it (not needed for act "none").  dx_add: [..., K], added to dx (the
    residual branch, or another projection of x).  grads: optional (dx, dw, db) to fill; an entry
    None is not computed.  dx may be ``dx_add`` itself.
    """
    torch = torch_()
    code, M, N, K = _rows(x, w)
    if act not in ACT_CODES:
        _act(act)
    need("dy", dy, x.shape[:-1] + (N,), x.dtype, x.device)
    if z is not None:
        need("z", z, dy.shape, x.dtype, x.device)
    elif act != "none":
        raise ValueError("z, the value before the activation, is needed for act %r" % (act,))
    if dx_add is not None:
        need("dx_add", dx_add, x.shape, x.dtype, x.device)
    if grads is None:
        grads = (made(stream, x.device, lambda: torch.empty_like(x)),
                 made(stream, x.device, lambda: torch.empty_like(w)),
                 made(stream, x.device,
                      lambda: torch.empty((N,), dtype=torch.float32, device=x.device)))
    dx, dw, db = grads
    for name, t, like, dt in (("dx", dx, x.shape, x.dtype), ("dw", dw, w.shape, x.dtype),
                              ("db", db, (N,), torch.float32)):
        if t is not None:
            need(name, t, like, dt, x.device)
    act = _act(act)
    size = nbytes("hyena_proj_bwd_workspace_bytes", M, N, K, act, code)
    ws, nws, _buf = workspace_of(workspace, size, x.device, stream)
    run("hyena_proj_bwd", x.device, x.data_ptr(), w.data_ptr(), ptr(z), dy.data_ptr(),
        ptr(dx_add), ptr(dx), ptr(dw), ptr(db), M, N, K, act, code, ws, nws,
        stream_handle(x.device, stream))
    return dx, dw, db
