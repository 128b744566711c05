"""Workloads of the gated linear recurrence and of the projections around a sequence mixer.

Two operators, each in every form that a user of the framework calls:

* the recurrence  x_t = k_t v_t,  s_t = exp(g_t) s_{t-1} + x_t,  y_t = q_t s_t  over [B, L, D], the
  log decay g given per token and group of d_g channels: forward ("scan"), forward and backward of
  a training step ("scan_train"), one token for a batch of running sequences ("scan_step");
* the projection  y = act(x W^T + bias) + residual: forward ("proj"; few rows are single tokens,
  many are prompts and training batches) and backward ("proj_bwd").

``own`` false: ``run`` computes them with elementary torch operations in fp32.  ``own`` true: with
the framework's kernels.  ``exact`` evaluates the definitions in fp64.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_MAX_ELEMS = 1 << 25   # B L D of the largest recurrence below
_MAX_MACS = 1 << 37    # M N K of the largest projection below


# ------------------------------------------------------------------------------------- cases
def _scan(name, op, B, L, D, d_g, dtype, s0=False, resets=False):
    c = {"op": op, "B": B, "L": L, "D": D, "d_g": d_g, "dtype": dtype, "s0": s0,
         "resets": resets}
    return dict(c, name=name) if name else c


def _proj(name, op, M, N, K, act, dtype, bias=True, residual=False):
    c = {"op": op, "M": M, "N": N, "K": K, "act": act, "dtype": dtype, "bias": bias,
         "residual": residual}
    return dict(c, name=name) if name else c


def listed():
    return [
        # a whole prompt through one layer, one decay for each group of 64 channels
        _scan("scan_prompt", "scan", 1, 8192, 4096, 64, "bf16"),
        # a long sequence in a narrow layer, one decay per channel, continued from a state
        _scan("scan_long_narrow", "scan", 1, 65536, 500, 1, "bf16", s0=True),
        # the smallest configuration, fp32: latency counts
        _scan("scan_tiny", "scan", 1, 1024, 64, 16, "f32"),
        # a training step of the wide layer
        _scan("train_wide", "scan_train", 1, 8192, 4096, 64, "bf16"),
        # a training step on packed documents (resets) with a decay per channel, odd sizes, fp32
        _scan("train_packed_f32", "scan_train", 3, 1537, 1000, 1, "f32", s0=True, resets=True),
        # one token for a full serving batch
        _scan("step_batch", "scan_step", 256, 1, 4096, 64, "bf16", s0=True),
        # one token for one sequence, a decay per channel
        _scan("step_one", "scan_step", 1, 1, 4096, 1, "bf16", s0=True),
        # output projection of a prompt: bias and the residual stream
        _proj("proj_prompt", "proj", 8192, 4096, 4096, "none", "bf16", residual=True),
        # one token for a few sequences: the weights' bytes are the whole cost
        _proj("proj_tokens", "proj", 8, 4096, 4096, "logsigmoid", "bf16"),
        # odd sizes in fp32
        _proj("proj_ragged_f32", "proj", 1001, 515, 770, "gelu", "f32", residual=True),
        # backward of a training batch's projection
        _proj("bwd_train", "proj_bwd", 8192, 4096, 4096, "silu", "bf16"),
        # backward of a narrow gate projection, ragged
        _proj("bwd_gate", "proj_bwd", 3000, 72, 1024, "logsigmoid", "bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_train", "scan_step", "proj", "proj", "proj_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("proj", "proj_bwd"):
        M, N, K = _log_int(rng, 1, 8192), _log_int(rng, 16, 4096), _log_int(rng, 16, 4096)
        if rng.random() < 0.6:  # most layers' widths are multiples of 64
            N, K = max(64, N // 64 * 64), max(64, K // 64 * 64)
        while M * N * K > (_MAX_MACS if dtype == "bf16" else _MAX_MACS >> 2):
            M = M // 2 + 1
        return _proj(None, op, M, N, K,
                     rng.choice(["none", "gelu", "silu", "sigmoid", "logsigmoid"]), dtype,
                     bias=rng.random() < 0.7, residual=op == "proj" and rng.random() < 0.5)
    d_g = rng.choice([1, 1, 2, 8, 16, 64, 64])
    D = d_g * max(1, _log_int(rng, 16, 4096) // d_g)
    if op == "scan_step":
        B, L = _log_int(rng, 1, 512), 1
    else:
        B, L = _log_int(rng, 1, 8), _log_int(rng, 1, 65536)
        while B * L * D > _MAX_ELEMS:
            if B > 1:
                B //= 2
            else:
                L = L // 2 + 1
    return _scan(None, op, B, L, D, d_g, dtype, s0=op == "scan_step" or rng.random() < 0.5,
                 resets=rng.random() < 0.3)


# ------------------------------------------------------------------------------------- inputs
def _inputs(case, seed):
    """The case's tensors on the GPU, from the seed alone."""
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 17)
    dt = _DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    if case["op"] in ("proj", "proj_bwd"):
        M, N, K = case["M"], case["N"], case["K"]
        s = {"x": randn(M, K).to(dt), "w": (randn(N, K) / math.sqrt(K)).to(dt), "bias": None,
             "residual": None}
        if case["bias"]:
            s["bias"] = 0.5 * randn(N)
        if case["residual"]:
            s["residual"] = randn(M, N).to(dt)
        if case["op"] == "proj_bwd":
            s["dy"] = randn(M, N).to(dt)
            s["z"] = None
            if case["act"] != "none":  # as the forward of the training step left it
                z = s["x"].float() @ s["w"].float().t()
                s["z"] = (z if s["bias"] is None else z + s["bias"]).to(dt)
        return s
    B, L, D, d_g = case["B"], case["L"], case["D"], case["d_g"]
    G = D // d_g
    # decays exp(g) between about 0.5 and 0.998, a level for each group and a part of each token
    level = torch.exp(torch.empty(G, device="cuda").uniform_(math.log(0.002), math.log(0.7),
                                                             generator=gen))
    s = {"q": randn(B, L, D).to(dt), "k": randn(B, L, D).to(dt), "v": randn(B, L, D).to(dt)}
    s["g"] = (-level * torch.exp(0.5 * randn(B, L, G))).to(dt)
    if case["resets"]:  # first tokens of packed documents forget the state
        first = torch.rand((B, L), generator=gen, device="cuda") < 4.0 / max(L, 16)
        s["g"][first] = -math.inf
    s["s0"] = randn(B, D) if case["s0"] else None
    if case["op"] == "scan_train":
        s["dy"] = randn(B, L, D).to(dt)
        s["ds"] = randn(B, D)
    if case["op"] == "scan_step":
        s["q"], s["k"], s["v"], s["g"] = (s[n][:, 0].contiguous() for n in "qkvg")
    return s


def prepare(case, seed):
    return dict(_inputs(case, seed), case=case)


# ------------------------------------------------------------------------------------- plain form
def _plain_scan(a, x, s0):
    """s_t = a_t s_{t-1} + x_t along dim 1 by doubling: after the step of span d, s holds the sum
    over the last 2 d terms and p the product of their decays."""
    s, p, d, L = x, a, 1, x.shape[1]
    while d < L:
        s = torch.cat((s[:, :d], s[:, d:] + p[:, d:] * s[:, :-d]), 1)
        p = torch.cat((p[:, :d], p[:, d:] * p[:, :-d]), 1)
        d *= 2
    return s if s0 is None else s + p * s0[:, None]


def _wide(g, d_g):
    return g.float().exp().repeat_interleave(d_g, -1) if d_g > 1 else g.float().exp()


def _groups(t, d_g):
    return t.reshape(*t.shape[:-1], -1, d_g).sum(-1)


def _act(z, act):
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    if act == "logsigmoid":
        return z.clamp(max=0) - torch.log1p(torch.exp(-z.abs()))
    return z


def _act_grad(z, act):
    if act == "gelu":
        return (0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    p = 1 / (1 + torch.exp(-z))
    if act == "silu":
        return p * (1 + z * (1 - p))
    if act == "sigmoid":
        return p * (1 - p)
    return 1 - p  # logsigmoid


def _plain(s):
    case = s["case"]
    op, dt = case["op"], _DTYPES[case["dtype"]]
    if op == "proj":
        z = s["x"].float() @ s["w"].float().t()
        if s["bias"] is not None:
            z = z + s["bias"]
        y = _act(z, case["act"])
        return (y if s["residual"] is None else y + s["residual"].float()).to(dt)
    if op == "proj_bwd":
        dz = s["dy"].float()
        if case["act"] != "none":
            dz = dz * _act_grad(s["z"].float(), case["act"])
        return {"dx": (dz @ s["w"].float()).to(dt), "dw": (dz.t() @ s["x"].float()).to(dt),
                "db": dz.sum(0)}
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    a = _wide(s["g"], case["d_g"])
    if op == "scan_step":
        state = a * s["s0"] + k * v
        return {"y": (q * state).to(dt), "state": state}
    st = _plain_scan(a, k * v, s["s0"])
    out = {"y": (q * st).to(dt), "state": st[:, -1]}
    if op == "scan":
        return out
    dy = s["dy"].float()
    u = q * dy
    u[:, -1] += s["ds"]
    # u_t += a_{t+1} u_{t+1}: the same recurrence backwards in time
    a_next = torch.cat((a[:, 1:], torch.zeros_like(a[:, :1])), 1)
    u = _plain_scan(a_next.flip(1), u.flip(1), None).flip(1)
    first = torch.zeros_like(st[:, :1]) if s["s0"] is None else s["s0"][:, None]
    dg = a * torch.cat((first, st[:, :-1]), 1) * u
    out.update(dq=(dy * st).to(dt), dk=(u * v).to(dt), dv=(u * k).to(dt),
               dg=_groups(dg, case["d_g"]).to(dt), ds0=a[:, 0] * u[:, 0])
    return out


# ------------------------------------------------------------------------------------- the kernels
def _kernels(s):
    import gated_causal_fir_b200 as fir

    case = s["case"]
    op = case["op"]
    if op == "proj":
        return fir.hyena_proj_fwd(s["x"], s["w"], s["bias"], act=case["act"],
                                  residual=s["residual"])
    if op == "proj_bwd":
        dx, dw, db = fir.hyena_proj_bwd(s["x"], s["w"], s["dy"], z=s["z"], act=case["act"])
        return {"dx": dx, "dw": dw, "db": db}
    q, k, v, g, s0, d_g = s["q"], s["k"], s["v"], s["g"], s["s0"], case["d_g"]
    if op == "scan_step":
        y, state = fir.hyena_scan_step(q, k, v, g, s0, d_g, state_out=torch.empty_like(s0))
        return {"y": y, "state": state}
    if op == "scan":
        y, state = fir.hyena_scan_fwd(q, k, v, g, d_g, s0=s0)
        return {"y": y, "state": state}
    ckpt = fir.hyena_scan_ckpt(q)
    y, state = fir.hyena_scan_fwd(q, k, v, g, d_g, s0=s0, ckpt=ckpt)
    dq, dk, dv, dg, ds0 = fir.hyena_scan_bwd(q, k, v, g, s["dy"], d_g, s0=s0, ds_out=s["ds"],
                                             ckpt=ckpt)
    return {"y": y, "state": state, "dq": dq, "dk": dk, "dv": dv, "dg": dg, "ds0": ds0}


def run(state):
    return _kernels(state) if own else _plain(state)


# ------------------------------------------------------------------------------------- cost, truth
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("proj", "proj_bwd"):
        M, N, K = case["M"], case["N"], case["K"]
        if case["op"] == "proj":
            return {"bytes": e * (M * K + N * K + M * N * (2 if case["residual"] else 1))
                    + (4 * N if case["bias"] else 0), "flops": 2 * M * N * K}
        return {"bytes": e * (2 * M * K + 2 * N * K + M * N * (1 if case["act"] == "none" else 2))
                + 4 * N, "flops": 4 * M * N * K}
    n, m = case["B"] * case["L"] * case["D"], case["B"] * case["L"] * case["D"] // case["d_g"]
    st = 4 * case["B"] * case["D"]
    states = st * (2 if case["s0"] else 1)
    if case["op"] == "scan_train":  # q, k, v, dy, g in; y, dq, dk, dv, dg out; s0, ds; state, ds0
        return {"bytes": e * (8 * n + 2 * m) + states + 2 * st, "flops": 15 * n}
    return {"bytes": e * (4 * n + m) + states, "flops": 4 * n}


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op in ("proj", "proj_bwd"):
        def curve(z):
            if case["act"] == "none":
                return z
            if case["act"] == "gelu":
                return z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
            if case["act"] == "silu":
                return z * torch.sigmoid(z)
            if case["act"] == "sigmoid":
                return torch.sigmoid(z)
            return -torch.logaddexp(torch.zeros_like(z), -z)

        if op == "proj":
            z = torch.mm(s["x"].double(), s["w"].double().t())
            y = curve(z + s["bias"].double() if s["bias"] is not None else z)
            return y + s["residual"].double() if s["residual"] is not None else y
        dz = s["dy"].double()
        if s["z"] is not None:
            z = s["z"].double().requires_grad_()
            dz, = torch.autograd.grad(curve(z), z, dz)
        return {"dx": torch.mm(dz, s["w"].double()), "dw": torch.mm(dz.t(), s["x"].double()),
                "db": dz.sum(0)}
    d_g = case["d_g"]
    q, k, v = (s[n].double() for n in "qkv")
    B, D = q.shape[0], q.shape[-1]
    decay = torch.exp(s["g"].double())
    state = s["s0"].double() if s["s0"] is not None else q.new_zeros(B, D)
    if op == "scan_step":
        state = state.view(B, -1, d_g) * decay[..., None]
        state = state.view(B, D) + k * v
        return {"y": q * state, "state": state}
    L = q.shape[1]
    x, before = k * v, torch.empty_like(q)
    for t in range(L):
        before[:, t] = state
        state = torch.addcmul(x[:, t].view(B, -1, d_g), state.view(B, -1, d_g),
                              decay[:, t, :, None]).view(B, D)
    states = torch.cat((before[:, 1:], state[:, None]), 1)
    out = {"y": q * states, "state": state}
    if op == "scan":
        return out
    dy, u, into = s["dy"].double(), s["ds"].double(), torch.empty_like(q)
    for t in range(L - 1, -1, -1):  # u: what reaches the state before token t + 1
        into[:, t] = torch.addcmul(u, q[:, t], dy[:, t])
        u = (into[:, t].view(B, -1, d_g) * decay[:, t, :, None]).view(B, D)
    dg = (before * into).view(B, L, -1, d_g).sum(-1) * decay
    out.update(dq=dy * states, dk=into * v, dv=into * k, dg=dg, ds0=u)
    return out
