"""Plain 64-bit forms of linear attention with a decay for each head and of the norms of queries and keys with their
rotation, on the CPU, and what their tests share.

Tolerances, in the 2-norm relative to the output's (`check` of gdr_testutil: no value further off than 8 times that
relative to the largest).  half(dtype) is half a step of the type: a result in bf16 has one rounding to it, its own.
What is computed on its way is carried in two bf16 planes, off by 2^-17 of the value, at most three of them on any path
(the products X Y^T, the state as an operand, Z in the state): 3 * 2^-17.  States take three planes (2^-25) and are
sums in fp32, as everything is for fp32 inputs: sums of up to 128 products behind one another on up to 6 levels,
each off by sqrt(128) half steps: 68, taken as 128 half steps of fp32.  dw is a sum over up to n tokens, n <= 512 here,
of differences of two such products whose errors do not cancel while the values do down to the size of one of
them: sqrt(2 n) = 32 times as much."""
from __future__ import annotations

import torch

from gdr_testutil import half, log_decay

SPLIT = 3 * 2.0 ** -17
F32 = 128 * 2.0 ** -24


def tol(name, dtype, per_head=False) -> float:
    if name in ("S", "dS0"):
        return F32
    if dtype == torch.float32:
        return 32 * F32 if name == "dw" else F32
    if name == "dw":
        return 32 * SPLIT + (0 if per_head else half(dtype))
    return half(dtype) + SPLIT


def rule(q, k, v, w, S0=None, lens=None, gate="bounded", scale=1.0):
    """The recurrence, token by token: (o, S_final); w [B,Hv,T] or [Hv]; lens divides T into packed sequences."""
    grp = v.shape[1] // q.shape[1]
    q, k = (x.repeat_interleave(grp, 1) for x in (q, k))
    a = torch.exp(log_decay(w, gate))
    if w.dim() == 1:
        a = a.view(1, -1, 1).expand(v.shape[:3])
    spans, at = ([(slice(None), 0, q.shape[2])] if lens is None else []), 0
    for n in lens or []:
        spans.append((slice(0, 1), at, at + n))
        at += n
    outs, finals = [], []
    for i, (rows, lo, hi) in enumerate(spans):
        S = v.new_zeros(v[rows].shape[0], v.shape[1], q.shape[3], v.shape[3])
        if S0 is not None:
            S = S0 if lens is None else S0[i:i + 1]
        for t in range(lo, hi):
            S = a[rows, :, t, None, None] * S + k[rows, :, t, :, None] * v[rows, :, t, None]
            outs.append(scale * (S * q[rows, :, t, :, None]).sum(-2))
        finals.append(S)
    o = torch.stack(outs, 2) if outs else v.new_zeros(v.shape[0], v.shape[1], 0, v.shape[3])
    return o, torch.cat(finals)


def make(B, T, Hk, Hv, dk, dv, dtype, gate="bounded", per_head=False, seed=0, states=0, layout="head"):
    """Seeded inputs on the CPU: q, k of unit length, v, w, dO and `states` states (0: None)."""
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    w = 2 * rn(B, T, Hv)
    d = dict(q=unit(rn(B, T, Hk, dk)), k=unit(rn(B, T, Hk, dk)), v=rn(B, T, Hv, dv),
             w=torch.nn.functional.logsigmoid(w + 2) if gate == "log" else w, dO=rn(B, T, Hv, dv))
    d = {n: x.to(dtype).transpose(1, 2) for n, x in d.items()}
    if layout == "head":
        d = {n: x.contiguous() for n, x in d.items()}
    if per_head:
        d["w"] = (-torch.exp2(-7 * torch.rand(Hv, generator=gen)) if gate == "log" else 2 * torch.randn(Hv, generator=gen)).float()
    for n in ("S0", "dS_final"):
        d[n] = (0.5 * rn(states, Hv, dk, dv)).float() if states else None
    return d


def reference(d, lens=None, gate="bounded", scale=1.0, grads=False):
    """o, S_final (and the gradients dq, dk, dv, dw, dS0 by automatic differentiation) in 64 bits."""
    names = ("q", "k", "v", "w", "S0")
    x = {n: d[n].double().requires_grad_(grads) if d[n] is not None else None for n in names}
    o, S = rule(*(x[n] for n in names), lens=lens, gate=gate, scale=scale)
    if not grads:
        return o, S
    n = o.shape[2]
    loss = (o * d["dO"].double()[:, :, :n]).sum()
    if d["dS_final"] is not None:
        loss = loss + (S * d["dS_final"].double()).sum()
    have = [n for n in names if x[n] is not None]
    g = torch.autograd.grad(loss, [x[n] for n in have], allow_unused=True)
    return o, S, {"d" + n: (gi if gi is not None else torch.zeros_like(x[n])) for n, gi in zip(have, g)}


def rotate(x, weight=None, positions=None, inv_freq=None, norm=True, interleaved=False, scale=1.0, eps=1e-6):
    """Norm and rotation of rows x [B,H,T,D]."""
    y = x
    if norm:
        y = y / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if weight is not None:
        y = y * weight
    if inv_freq is not None:
        R = 2 * inv_freq.shape[0]
        pos = positions if positions.dim() == 2 else positions[None]
        ang = pos.double()[:, None, :, None] * inv_freq.double()
        c, s = ang.cos(), ang.sin()
        if interleaved:
            a, b = y[..., 0:R:2], y[..., 1:R:2]
            turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
        else:
            a, b = y[..., :R // 2], y[..., R // 2:R]
            turned = torch.cat([a * c - b * s, b * c + a * s], -1)
        y = torch.cat([turned, y[..., R:]], -1)
    return scale * y
