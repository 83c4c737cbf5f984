"""Plain 64-bit forms of the head-gated delta rule and of the norms around a block, on the CPU, and what
the tests of both share.

Tolerances, in the 2-norm relative to the output's.  `half(dtype)` is half a step of the type relative to
the value: one rounding is off by at most that.  Every output in bf16 has one rounding to it, its own;
what is computed on its way is carried in two or three bf16 planes, which are off by 2^-17 and 2^-25 of the
value: at most 5 operands of two planes lie on any path (S, dS, F, dE, and dP or dA), so 5 * 2^-17 comes on top
(8 times as much for dw, a difference of sums), and is the whole tolerance of the fp32 states.
fp32: sums of up to 128 products, 6 of them one behind another, each off by sqrt(128) half steps: 68, taken
as 128; dw is a difference of such sums, 4 times as much."""
from __future__ import annotations

import torch

CHUNK = 64
ROUNDINGS = {"o": 1, "S": 0, "dq": 1, "dk": 1, "dv": 1, "dw": 1, "dbeta": 1, "dS0": 0}
SPLIT = 5 * 2.0 ** -17


def half(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def tol(name, dtype) -> float:
    if dtype == torch.float32:
        return 128 * half(dtype) * (4 if name == "dw" else 1)
    return ROUNDINGS[name] * half(dtype) + SPLIT * (8 if name == "dw" else 1)


def check(name, got, ref, t, more=0.0):
    """2-norm of the difference within t of the reference's, and no value further off than 8 t of the largest;
    `more` is added to both (the absolute error of terms that cancel)."""
    got, ref = got.detach().double().cpu(), ref.detach().double()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    if not ref.numel():
        return
    assert torch.isfinite(got).all(), f"{name}: {int((~torch.isfinite(got)).sum())} values are not finite"
    norm, d = float(ref.norm()), got - ref
    rel = float(d.norm()) / norm if norm else float(d.norm())
    big = float(d.abs().max()) / float(ref.abs().max()) if norm else float(d.abs().max())
    print(f"   {name}: off by {rel:.2e} (2-norm), {big:.2e} (largest), allowed {t:.2e}", flush=True)
    top = float(ref.abs().max())
    assert rel <= t + more / (norm or 1.0) and big <= 8 * t + more / (top or 1.0), (name, rel, big, t, more)


def log_decay(w, gate, g_min=-5.0):
    if gate == "log":
        return w
    return g_min * torch.sigmoid(w) if gate == "bounded" else -torch.nn.functional.softplus(w)


def rule(q, k, v, w, beta, S0=None, lens=None, gate="bounded", scale=1.0):
    """The recurrence, token by token: (o, S_final).  q, k [B,Hk,T,dk] and so on, any float type; lens
    divides T into packed sequences."""
    grp = v.shape[1] // q.shape[1]
    q, k = (x.repeat_interleave(grp, 1) for x in (q, k))
    a = torch.exp(log_decay(w, gate))
    spans = [(slice(None), 0, q.shape[2])] if lens is None else []
    at = 0
    for n in lens or []:
        spans.append((slice(0, 1), at, at + n))
        at += n
    outs, finals = [], []
    for i, (rows, lo, hi) in enumerate(spans):
        if S0 is not None:
            S = S0 if lens is None else S0[i:i + 1]
        else:
            S = v.new_zeros(v[rows].shape[0], v.shape[1], q.shape[3], v.shape[3])
        for t in range(lo, hi):
            kt = k[rows, :, t, :, None]
            S = a[rows, :, t, None, None] * S
            f = v[rows, :, t] - (S * kt).sum(-2)
            S = S + kt * (beta[rows, :, t, None] * f)[:, :, None]
            outs.append(scale * (S * q[rows, :, t, :, None]).sum(-2))
        finals.append(S)
    o = torch.stack(outs, 2) if outs else v.new_zeros(v.shape[0], v.shape[1], 0, v.shape[3])
    return o, torch.cat(finals)


def make(B, T, Hk, Hv, dk, dv, dtype, gate="bounded", seed=0, states=0, layout="head"):
    """Seeded inputs on the CPU: q, k of unit length, v, w, beta, dO and `states` states (0: None)."""
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    w = 2 * rn(B, T, Hv)
    d = dict(q=unit(rn(B, T, Hk, dk)), k=unit(rn(B, T, Hk, dk)), v=rn(B, T, Hv, dv),
             w=torch.nn.functional.logsigmoid(w + 2) if gate == "log" else w, beta=torch.sigmoid(rn(B, T, Hv)), dO=rn(B, T, Hv, dv))
    d = {n: x.to(dtype).transpose(1, 2) for n, x in d.items()}
    if layout == "head":
        d = {n: x.contiguous() for n, x in d.items()}
    for n in ("S0", "dS_final"):
        d[n] = (0.5 * rn(states, Hv, dk, dv)).float() if states else None
    return d


def reference(d, lens=None, gate="bounded", scale=1.0, grads=False):
    """o, S_final (and the gradients dq, dk, dv, dw, dbeta, dS0 by automatic differentiation) in 64 bits."""
    x = {n: d[n].double().requires_grad_(grads) if d[n] is not None else None for n in ("q", "k", "v", "w", "beta", "S0")}
    o, S = rule(*(x[n] for n in ("q", "k", "v", "w", "beta", "S0")), lens=lens, gate=gate, scale=scale)
    if not grads:
        return o, S
    n = o.shape[2]
    loss = (o * d["dO"].double()[:, :, :n]).sum()
    if d["dS_final"] is not None:
        loss = loss + (S * d["dS_final"].double()).sum()
    names = [n for n in ("q", "k", "v", "w", "beta", "S0") if x[n] is not None]
    g = torch.autograd.grad(loss, [x[n] for n in names], allow_unused=True)
    return o, S, {("dS0" if n == "S0" else "d" + n): (gi if gi is not None else torch.zeros_like(x[n])) for n, gi in zip(names, g)}


def gpu(d):
    """The inputs on the GPU, their memory order kept."""
    return {n: None if x is None else x.cuda() for n, x in d.items()}


def gate_args(gate):
    return {"bounded": dict(g_min=-5.0), "softplus": dict(g_min=-float("inf")), "log": dict(log_decay=True)}[gate]


def norms(x, weight=None, z=None, act="silu", residual=None, alpha=1.0, next_weight=None, eps=1e-6):
    """The norms around a block: (s, y)."""
    rms = lambda t: torch.sqrt((t * t).mean(-1, keepdim=True) + eps)  # noqa: E731
    h = x
    if weight is not None:
        h = h / rms(h) * weight
    if z is not None:
        h = h * (torch.sigmoid(z) if act == "sigmoid" else z * torch.sigmoid(z))
    s = alpha * h
    if residual is not None:
        s = s + residual
    return s, None if next_weight is None else s / rms(s) * next_weight
