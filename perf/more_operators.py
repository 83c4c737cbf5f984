"""Cases of linear attention with a decay for each head (chunked forward, its gradients, the recurrent step on
a pool of states) and of the norms of queries and keys with the rotation by position (forward, gradients), in a
plain form and through this package's entry points.

`own` False: elementary torch operations in 32 bits (in 64 for cumulative log-decays, for the decay's gradient,
sums of cancelling terms, and for the angles), rounded once at the end.  `own` True: the calls a user makes.

Linear attention with decay, per sequence and value head, with a state S (dk x dv) and one log-decay a token:
    S <- e^{g_t} S + k_t v_t^T;  o_t = scale S^T q_t
with g = g_min sigmoid(w), -softplus(w) or w itself, w being one value a token and head or one a head; value
head h reads query and key head h / (Hv / Hk).

Norm and rotation, per row x of D values at position p:
    n = x / rms(x) * weight;  y = scale * n with its first R values rotated in pairs by the angles p * inv_freq
where the norm, the weight or the rotation may be absent; pairs are (i, i + R/2) or (2i, 2i + 1).
"""
import math

import torch

own = False

CHUNK = 64
G_MIN = -5.0
EPS = 1e-6


def listed():
    """The cases by name."""
    return [
        # one short prompt of a small model: latency
        dict(name="fwd one prompt of 130", op="fwd", B=1, lens="", T=130, Hk=4, Hv=4, dk=128, dv=128, dtype="bf16", gate="head",
             layout="token", state=True),
        # a serving step's prompts packed one behind another: an empty one, one token, chunk borders, shared key heads
        dict(name="fwd packed prompts", op="fwd", B=1, lens="517,0,1,64,1300,63,65,2000,89", T=4099, Hk=8, Hv=16, dk=128, dv=128,
             dtype="bf16", gate="softplus", layout="fused", state=True),
        # one document of this repository's headline length and heads, a fixed decay for each head
        dict(name="fwd 64K tokens", op="fwd", B=1, lens="", T=65536, Hk=16, Hv=16, dk=128, dv=128, dtype="bf16", gate="head",
             layout="head", state=False),
        # fp32 inputs, an odd length and unequal head sizes
        dict(name="fwd fp32 1001", op="fwd", B=2, lens="", T=1001, Hk=4, Hv=8, dk=64, dv=32, dtype="f32", gate="log", layout="head",
             state=True),
        # the gradients of a training step at this repository's 4096-token batch
        dict(name="bwd 2x4096", op="bwd", B=2, lens="", T=4096, Hk=16, Hv=16, dk=128, dv=128, dtype="bf16", gate="bounded",
             layout="token", state=False),
        # fp32 gradients of packed documents with shared key heads, entering states and a learned decay a head
        dict(name="bwd fp32 packed", op="bwd", B=1, lens="300,1,0,447,64", T=812, Hk=2, Hv=4, dk=64, dv=128, dtype="f32",
             gate="head", layout="token", state=True),
        # one sequence that answers token by token
        dict(name="step 1 sequence", op="step", B=1, slots=4, pad=0, T=1, Hk=4, Hv=8, dk=128, dv=128, dtype="bf16", gate="bounded"),
        # a serving batch of 512 rows, some of them padding, over a larger pool
        dict(name="step 512 sequences", op="step", B=512, slots=528, pad=7, T=1, Hk=8, Hv=16, dk=128, dv=128, dtype="bf16",
             gate="head"),
        # queries and keys of three answering sequences, far into their contexts
        dict(name="rotate 3 tokens", op="rotate", dir="fwd", B=3, T=1, Hq=16, Hk=4, D=128, R=128, dtype="bf16", wdtype="bf16",
             norm=True, pairs="half", base=1000000.0, start=120000, layout="fused"),
        # a prefill's packed tokens, shared key heads
        dict(name="rotate 16K tokens", op="rotate", dir="fwd", B=1, T=16384, Hq=32, Hk=8, D=128, R=128, dtype="bf16", wdtype="bf16",
             norm=True, pairs="half", base=1000000.0, start=0, layout="fused"),
        # gradients at the 4096-token batch
        dict(name="rotate bwd 2x4096", op="rotate", dir="bwd", B=2, T=4096, Hq=16, Hk=16, D=128, R=64, dtype="bf16", wdtype="f32",
             norm=True, pairs="half", base=10000.0, start=0, layout="token"),
        # gradients in fp32 with a head size that is no power of two, neighbouring pairs, a part of the head rotated
        dict(name="rotate bwd fp32", op="rotate", dir="bwd", B=1, T=1003, Hq=5, Hk=1, D=80, R=36, dtype="f32", wdtype="f32",
             norm=True, pairs="near", base=10000.0, start=70, layout="head"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "step", "rotate", "rotate", "rotate"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "rotate":
        D = rng.choice([32, 64, 80, 96, 128, 192, 256])
        Hk = rng.choice([1, 2, 4, 8])
        Hq = Hk * rng.choice([1, 2, 4])
        most = (1 << 25) // (D * (Hq + Hk))
        B = rng.choice([1, 1, 2, 3])
        R = rng.choice([D, D, D // 2, 2 * rng.randrange(1, D // 2), 0])
        return dict(op=op, dir=rng.choice(["fwd", "bwd"]), B=B, T=max(1, _spread(rng, 1, most) // B), Hq=Hq, Hk=Hk, D=D, R=R,
                    dtype=dtype, wdtype=rng.choice([dtype, "f32", "none"]), norm=R == 0 or rng.random() < 0.8,
                    pairs=rng.choice(["half", "near"]), base=rng.choice([1e4, 1e6]), start=rng.choice([0, _spread(rng, 1, 1000000)]),
                    layout=rng.choice(["token", "head", "fused"]))
    Hk, grp = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4])
    case = dict(op=op, Hk=Hk, Hv=Hk * grp, dk=rng.choice([32, 64, 128]), dv=rng.choice([32, 64, 128]), dtype=dtype,
                gate=rng.choice(["bounded", "softplus", "log", "head"]))
    if op == "step":
        B = _spread(rng, 1, 256)
        return dict(case, B=B, slots=B + rng.randrange(0, 9), pad=rng.randrange(0, B) if rng.random() < 0.5 else 0, T=rng.choice([1, 1, 2, 5]))
    most = (20000 if op == "fwd" else 4000) // grp
    total = _spread(rng, 1, most)
    lens, B = "", 1
    if rng.random() < 0.5:
        cuts = sorted(rng.randrange(0, total + 1) for _ in range(rng.randrange(1, 9)))
        lens = ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [total]))
    else:
        B = rng.choice([1, 2, 3])
        total = max(1, total // B)
    return dict(case, B=B, lens=lens, T=total, layout=rng.choice(["token", "head", "fused"]), state=rng.random() < 0.5)


# ---------------------------------------------------------------------------------------------------------------- inputs

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _lens(case):
    return [int(n) for n in case["lens"].split(",")] if case["lens"] else [case["T"]] * case["B"]


def _unit(x):
    return x / x.double().square().sum(-1, keepdim=True).sqrt().clamp_min(1e-30)


def _arrange(tensors, layout):
    """[B, T, H, D] tensors as [B, H, T, D] views: in a token's order, in a head's, or columns of one projection's output."""
    if layout == "fused":
        x = torch.cat([t.flatten(2) for t in tensors], dim=-1)
        out, at = [], 0
        for t in tensors:
            n = t.shape[2] * t.shape[3]
            out.append(x[..., at:at + n].unflatten(-1, t.shape[2:]).transpose(1, 2))
            at += n
        return out
    out = [t.transpose(1, 2) for t in tensors]
    return [t.contiguous() for t in out] if layout == "head" else out


def prepare(case, seed):
    """The inputs, on the GPU, from the seed alone."""
    dev = _device()
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    dt = _TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    st = {"case": case}
    if case["op"] == "rotate":
        B, T, Hq, Hk, D, R = (case[n] for n in ("B", "T", "Hq", "Hk", "D", "R"))
        row = lambda H: (normal(B, T, H, D) * torch.exp(0.5 * normal(B, T, H, 1))).to(dt)  # noqa: E731
        extra = [normal(B, T, Hk, D).to(dt)] if case["layout"] == "fused" else []      # the values beside them
        st["q"], st["k"] = _arrange([row(Hq), row(Hk)] + extra, case["layout"])[:2]
        wt = _TYPES.get(case["wdtype"])
        st["q_weight"], st["k_weight"] = ((1 + 0.1 * normal(D)).to(wt) if wt is not None and case["norm"] else None for _ in "qk")
        # rows of a batch are at places of their own
        st["positions"] = (torch.arange(T, device=dev) + case["start"] + 13 * torch.arange(B, device=dev)[:, None]).to(torch.int32) if R else None
        st["inv_freq"] = (case["base"] ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)).float().to(dev) if R else None
        st["q_scale"], st["k_scale"] = D ** -0.5, 1.0
        if case["dir"] == "bwd":
            st["dq"], st["dk"] = _arrange([normal(B, T, Hq, D).to(dt), normal(B, T, Hk, D).to(dt)], "token" if case["layout"] != "head" else "head")
        return st
    B, T, Hk, Hv, dk, dv = (case[n] for n in ("B", "T", "Hk", "Hv", "dk", "dv"))
    q, k, v = _unit(normal(B, T, Hk, dk)).to(dt), _unit(normal(B, T, Hk, dk)).to(dt), normal(B, T, Hv, dv).to(dt)
    st["q"], st["k"], st["v"] = _arrange([q, k, v], case.get("layout", "head"))
    if case["gate"] == "head":   # the heads' memories grow from one token to some hundred
        st["w"] = -torch.exp2(-8.0 * torch.rand(Hv, generator=gen, device=dev))
    else:
        w = 2 * normal(B, T, Hv)
        w = (torch.nn.functional.logsigmoid(w + 2) if case["gate"] == "log" else w).to(dt).transpose(1, 2)
        st["w"] = w.contiguous() if case.get("layout", "head") == "head" else w
    st["scale"] = dk ** -0.5
    if case["op"] == "step":
        st["S"] = 0.5 * normal(case["slots"], Hv, dk, dv)
        order = torch.randperm(case["slots"], generator=torch.Generator().manual_seed(int(seed)))[:B].to(torch.int32)
        if case["pad"]:
            order[B - case["pad"]:] = -1
        st["slots"] = order.to(dev)
        return st
    lens = _lens(case)
    st["t_max"] = max(lens)
    st["cu_seqlens"] = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).to(torch.int32).to(dev) if case["lens"] else None
    st["S0"] = 0.3 * normal(len(lens), Hv, dk, dv) if case["state"] else None
    if case["op"] == "bwd":
        dO = normal(B, T, Hv, dv).to(dt).transpose(1, 2)
        st["dO"] = dO.contiguous() if case["layout"] == "head" else dO
        st["dS_final"] = 0.3 * normal(len(lens), Hv, dk, dv) if case["state"] else None
    return st


# ------------------------------------------------------------------------------------------------------------ plain forms


def _gate(w, gate):
    """The log-decay and its derivative by w."""
    if gate in ("log", "head"):
        return w, torch.ones_like(w)
    s = 1 / (1 + torch.exp(-w))
    if gate == "bounded":
        return G_MIN * s, G_MIN * s * (1 - s)
    return -(torch.clamp_min(w, 0) + torch.log1p(torch.exp(-w.abs()))), -s


def _tokens_w(st):
    """w of every token, [B, Hv, T]."""
    c, w = st["case"], st["w"]
    return w[None, :, None].expand(c["B"], c["Hv"], c["T"]) if c["gate"] == "head" else w


def _pad(x, st):
    """[B, H, T, ...] tokens as [sequences, H, whole chunks, ...], zeros behind each sequence's end."""
    cu, n = st["cu_seqlens"], -(-st["t_max"] // CHUNK) * CHUNK
    if cu is None:
        B, H, T = x.shape[:3]
        y = x.new_zeros((B, H, n) + x.shape[3:])
        y[:, :, :T] = x
        return y
    at = torch.arange(n, device=x.device) + cu[:-1, None]
    y = x[0][:, at.clamp_max(x.shape[2] - 1)].transpose(0, 1)
    keep = (at < cu[1:, None]).view((at.shape[0], 1, n) + (1,) * (y.dim() - 3))
    return torch.where(keep, y, torch.zeros((), dtype=y.dtype, device=y.device))


def _unpad(y, st):
    """The inverse of _pad."""
    cu, T = st["cu_seqlens"], st["q"].shape[2]
    if cu is None:
        return y[:, :, :T]
    t = torch.arange(T, device=y.device)
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return y[seq, :, t - cu[seq].long()].transpose(0, 1)[None]


def _chunks(st):
    """What both directions of the chunk form start with, per sequence, value head and chunk of 64 tokens."""
    c = st["case"]
    grp = c["Hv"] // c["Hk"]
    p = {}
    for n in ("q", "k", "v"):
        x = _pad(st[n], st).float().unflatten(2, (-1, CHUNK))
        p[n] = x.repeat_interleave(grp, 1) if n != "v" else x
    w = _pad(_tokens_w(st), st).double()
    g, p["dgate"] = _gate(w, c["gate"])
    at = torch.arange(w.shape[2], device=w.device)
    if st["cu_seqlens"] is None:
        live = (at < st["t_max"]).expand_as(w)
    else:
        cu = st["cu_seqlens"]
        live = (at[None, None] < (cu[1:] - cu[:-1])[:, None, None]).expand_as(w)
    p["live"] = live
    G = torch.where(live, g, 0.0).unflatten(2, (-1, CHUNK)).cumsum(-1)
    p["D"] = torch.exp((G[..., :, None] - G[..., None, :]).tril()).float().tril()
    p["gam"], p["eta"], p["last"] = G.exp().float()[..., None], (G[..., -1:] - G).exp().float()[..., None], G[..., -1].exp().float()[..., None, None]
    Keta = (p["eta"] * p["k"]).transpose(-1, -2)
    n, H, nc = p["v"].shape[:3]
    S = st["S0"].clone() if st["S0"] is not None else p["v"].new_zeros(n, H, c["dk"], c["dv"])
    states = []
    for i in range(nc):
        states.append(S)
        S = p["last"][:, :, i] * S + Keta[:, :, i] @ p["v"][:, :, i]
    p["S"], p["S_final"] = torch.stack(states, 2), S
    return p


def _plain_fwd(st):
    p = _chunks(st)
    o = p["gam"] * (p["q"] @ p["S"]) + (p["q"] @ p["k"].transpose(-1, -2) * p["D"]) @ p["v"]
    return _unpad((st["scale"] * o).flatten(2, 3), st).to(st["v"].dtype), p["S_final"]


def _plain_bwd(st):
    c = st["case"]
    p = _chunks(st)
    T_ = lambda x: x.transpose(-1, -2)  # noqa: E731
    k, q, v, S, gam, eta = p["k"], p["q"], p["v"], p["S"], p["gam"], p["eta"]
    dO = st["scale"] * _pad(st["dO"], st).float().unflatten(2, (-1, CHUNK))
    Qgam = T_(gam * q)
    dS = st["dS_final"].clone() if st["dS_final"] is not None else torch.zeros_like(S[:, :, 0])
    nc = S.shape[2]
    dSs = [None] * nc
    for i in reversed(range(nc)):
        dSs[i] = dS
        dS = p["last"][:, :, i] * dS + Qgam[:, :, i] @ dO[:, :, i]
    dSn = torch.stack(dSs, 2)
    QK, OV = T_(q @ T_(k) * p["D"]), dO @ T_(v) * p["D"]
    dq_ = gam * (dO @ T_(S)) + OV @ k
    behind = eta * (v @ T_(dSn))
    dk_ = behind + T_(OV) @ q
    dv_ = eta * (k @ dSn) + QK @ dO
    # the log-decay's gradient: cancelling terms, summed in 64 bits
    dG = (q.double() * dq_ - k.double() * dk_).sum(-1)
    dG[..., -1] += (k.double() * behind).sum((-1, -2)) + (p["last"].double() * S * dSn).sum((-1, -2))
    dg = dG.flip(-1).cumsum(-1).flip(-1).flatten(2, 3) * p["dgate"]
    n, _, _, C, dk = dq_.shape
    heads = lambda x: x.view(n, c["Hk"], -1, nc, C, dk).sum(2)  # noqa: E731  value heads that share a key head
    out = [_unpad(x.flatten(2, 3).to(st["q"].dtype), st) for x in (heads(dq_), heads(dk_), dv_)]
    if c["gate"] == "head":
        out.append((dg * p["live"]).sum((0, 2)).to(st["w"].dtype))
    else:
        out.append(_unpad(dg.to(st["w"].dtype), st))
    return tuple(out) + ((dS,) if st["S0"] is not None else ())


def _plain_step(st):
    c = st["case"]
    grp = c["Hv"] // c["Hk"]
    at = st["slots"].long()
    keep = (at >= 0)[:, None, None, None]
    S = st["S"][at.clamp_min(0)]
    q, k, v = st["q"].float().repeat_interleave(grp, 1), st["k"].float().repeat_interleave(grp, 1), st["v"].float()
    a = torch.exp(_gate(_tokens_w(st).float(), c["gate"])[0])
    outs = []
    for t in range(c["T"]):
        S = a[:, :, t, None, None] * S + k[:, :, t, :, None] * v[:, :, t, None]
        outs.append(st["scale"] * (S * q[:, :, t, :, None]).sum(-2))
    # padding rows go to a row behind the pool, which is dropped
    pool = torch.cat([st["S"], torch.zeros_like(st["S"][:1])])
    pool[torch.where(at >= 0, at, st["S"].shape[0])] = S
    st["S"].copy_(pool[:-1])
    return torch.where(keep, torch.stack(outs, 2), 0.0).to(st["v"].dtype), st["S"]


def _turn(x, st, sign):
    """The first R values of each row rotated by sign * position * inv_freq."""
    R = st["case"]["R"]
    if not R:
        return x
    ang = sign * st["positions"].double()[:, None, :, None] * st["inv_freq"].double()     # [B, 1, T, R/2]
    c, s = ang.cos().float(), ang.sin().float()
    y = x.clone()
    if st["case"]["pairs"] == "half":
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y[..., :R // 2], y[..., R // 2:R] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y[..., 0:R:2], y[..., 1:R:2] = a * c - b * s, b * c + a * s
    return y


def _plain_rotate(st):
    case, outs = st["case"], []
    for n in "qk":
        x = st[n].float()
        w = st[n + "_weight"].float() if st[n + "_weight"] is not None else 1.0
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) if case["norm"] else 1.0
        if case["dir"] == "fwd":
            outs.append((st[n + "_scale"] * _turn(x * r * w, st, 1.0)).to(st[n].dtype))
            continue
        dn = _turn(st[n + "_scale"] * st["d" + n].float(), st, -1.0)
        xh, t = x * r, dn * w
        dx = r * (t - xh * (t * xh).mean(-1, keepdim=True)) if case["norm"] else t
        outs.append(dx.to(st[n].dtype))
        if st[n + "_weight"] is not None:
            outs.append((dn * xh).sum((0, 1, 2)).to(st[n + "_weight"].dtype))
    return tuple(outs)


# ------------------------------------------------------------------------------------------------------------------- run


def _gate_args(case):
    return {"bounded": dict(g_min=G_MIN), "softplus": dict(g_min=-math.inf), "log": dict(log_decay=True), "head": dict(log_decay=True)}[case["gate"]]


def run(state):
    """One pass through the operator."""
    st, c = state, state["case"]
    if not own:
        return {"fwd": _plain_fwd, "bwd": _plain_bwd, "step": _plain_step, "rotate": _plain_rotate}[c["op"]](st)
    import chunked_gated_delta_amd as kda
    if c["op"] == "rotate":
        args = dict(q_weight=st["q_weight"], k_weight=st["k_weight"], positions=st["positions"], inv_freq=st["inv_freq"], norm=c["norm"],
                    interleaved=c["pairs"] == "near", q_scale=st["q_scale"], k_scale=st["k_scale"], eps=EPS)
        if c["dir"] == "fwd":
            return kda.qk_norm_rope_fwd(st["q"], st["k"], **args)
        dq, dk, dqw, dkw = kda.qk_norm_rope_bwd(st["q"], st["k"], st["dq"], st["dk"], **args)
        return (dq, dk) if dqw is None else (dq, dqw, dk, dkw)
    args = [st[n] for n in ("q", "k", "v", "w")]
    kw = dict(scale=st["scale"], **_gate_args(c))
    if c["op"] == "step":
        return kda.lad_decode(*args, st["S"], st["slots"], **kw), st["S"]
    if c["op"] == "fwd":
        return kda.lad_chunk_fwd(*args, st["S0"], cu_seqlens=st["cu_seqlens"], **kw)
    out = kda.lad_chunk_bwd(*args, st["dO"], st["S0"], st["dS_final"], cu_seqlens=st["cu_seqlens"], want_dS0=st["S0"] is not None, **kw)
    return out if st["S0"] is not None else out[:4]


# ------------------------------------------------------------------------------------------- the definition, in 64 bits


def exact(case, seed):
    """run()'s answer from the token recurrence (and its adjoint), and from the norm's definition, in 64 bits."""
    st = prepare(case, seed)
    return {"rotate": _exact_rotate, "step": _exact_step}.get(case["op"], _exact_rule)(st)


def _exact_gate(st):
    """Log-decay and its derivative, [B, Hv, T]."""
    c = st["case"]
    w = st["w"].double()
    if c["gate"] == "head":
        w = w.view(1, -1, 1).expand(c["B"], -1, c["T"])
    if c["gate"] == "bounded":
        return G_MIN * torch.sigmoid(w), G_MIN * torch.sigmoid(w) * torch.sigmoid(-w)
    if c["gate"] == "softplus":
        return torch.nn.functional.logsigmoid(-w), -torch.sigmoid(w)
    return w, torch.ones_like(w)


def _exact_rule(st):
    c, grp = st["case"], st["case"]["Hv"] // st["case"]["Hk"]
    ends = st["cu_seqlens"].tolist() if st["cu_seqlens"] is not None else None
    g, dgate = _exact_gate(st)
    a = g.exp()
    q, k = (st[n].double().repeat_interleave(grp, 1) for n in ("q", "k"))
    v, bwd = st["v"].double(), c["op"] == "bwd"
    o = torch.zeros_like(v)
    dq, dk, dv, dg = (torch.zeros_like(x) for x in (q, k, v, g))
    dO = st["scale"] * st["dO"].double() if bwd else None
    finals, starts = [], []
    spans = [(slice(None), 0, c["T"], slice(None))] if ends is None else [(slice(0, 1), a_, b_, slice(i, i + 1)) for i, (a_, b_) in enumerate(zip(ends, ends[1:]))]
    for rows, lo, hi, at in spans:
        n = c["B"] if ends is None else 1
        S = st["S0"][at].double() if st["S0"] is not None else v.new_zeros(n, c["Hv"], c["dk"], c["dv"])
        kept = []
        for t in range(lo, hi):
            old = a[rows, :, t, None, None] * S
            S = old + k[rows, :, t, :, None] * v[rows, :, t, None]
            if bwd:
                kept.append(old)
                dq[rows, :, t] = (S * dO[rows, :, t, None]).sum(-1)
            else:
                o[rows, :, t] = st["scale"] * (S * q[rows, :, t, :, None]).sum(-2)
        finals.append(S)
        if not bwd:
            continue
        R = st["dS_final"][at].double() if st["dS_final"] is not None else torch.zeros_like(S)
        for t in reversed(range(lo, hi)):
            R = R + q[rows, :, t, :, None] * dO[rows, :, t, None]
            dk[rows, :, t], dv[rows, :, t] = (R * v[rows, :, t, None]).sum(-1), (R * k[rows, :, t, :, None]).sum(-2)
            dg[rows, :, t] = (R * kept.pop()).sum((-1, -2))
            R = a[rows, :, t, None, None] * R
        starts.append(R)
    if not bwd:
        return o, torch.cat(finals)
    shared = lambda x: x.unflatten(1, (c["Hk"], grp)).sum(2)  # noqa: E731
    dw = dg * dgate
    out = (shared(dq), shared(dk), dv, dw.sum((0, 2)) if c["gate"] == "head" else dw)
    return out + ((torch.cat(starts),) if st["S0"] is not None else ())


def _exact_step(st):
    c, grp = st["case"], st["case"]["Hv"] // st["case"]["Hk"]
    o, pool = torch.zeros_like(st["v"], dtype=torch.float64), st["S"]
    at = st["slots"].long()
    rows = (at >= 0).nonzero()[:, 0]
    S = pool[at[rows]].double()
    q, k = (st[n][rows].double().repeat_interleave(grp, 1) for n in ("q", "k"))
    v, a = st["v"][rows].double(), _exact_gate(st)[0][rows].exp()
    for t in range(c["T"]):
        S = S * a[:, :, t, None, None] + k[:, :, t, :, None] * v[:, :, t, None]
        o[rows, :, t] = st["scale"] * (q[:, :, t, None] @ S)[:, :, 0]
    pool = pool.double()
    pool[at[rows]] = S
    return o, pool


def _exact_rotate(st):
    """Rotation as a product of complex numbers; gradients by automatic differentiation of the definition."""
    case, outs = st["case"], []
    R, D = case["R"], case["D"]
    for n in "qk":
        x = st[n].double().requires_grad_()
        w = st[n + "_weight"].double().requires_grad_() if st[n + "_weight"] is not None else None
        y = x
        if case["norm"]:
            y = y / (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt()
        if w is not None:
            y = y * w
        if R:
            turn = torch.polar(torch.ones(1, dtype=torch.float64, device=x.device), st["positions"].double()[:, None, :, None] * st["inv_freq"].double())
            pair = y[..., :R].unflatten(-1, (2, R // 2)).transpose(-1, -2) if case["pairs"] == "half" else y[..., :R].unflatten(-1, (R // 2, 2))
            z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
            z = z.transpose(-1, -2) if case["pairs"] == "half" else z
            y = torch.cat([z.flatten(-2), y[..., R:]], -1)
        y = st[n + "_scale"] * y
        if case["dir"] == "fwd":
            outs.append(y.detach())
        else:
            outs += torch.autograd.grad(y, [x] + ([w] if w is not None else []), st["d" + n].double())
    return tuple(outs)


# ------------------------------------------------------------------------------------------------------------------ work


def work(case):
    """Bytes read and written once each, and the recurrence's multiplications and additions."""
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rotate":
        n = case["B"] * case["T"] * (case["Hq"] + case["Hk"]) * case["D"]
        bwd = case["dir"] == "bwd"
        weights = 2 * case["D"] * {"bf16": 2, "f32": 4, "none": 0}[case["wdtype"]] * case["norm"]
        return {"bytes": n * e * (3 if bwd else 2) + weights * (2 if bwd else 1) + (4 * case["B"] * case["T"] + 2 * case["R"]) * (case["R"] > 0),
                "flops": n * ((10 if bwd else 4) * case["norm"] + 3 * (case["R"] > 0) + 1)}
    Hk, Hv, dk, dv, B, T = (case[n] for n in ("Hk", "Hv", "dk", "dv", "B", "T"))
    head = case["gate"] == "head"
    rows = (B - case["pad"] if case["op"] == "step" else B) * T
    tok = rows * (2 * Hk * dk + Hv * dv + (0 if head else Hv)) * e + (4 * Hv if head else 0)      # q, k, v, w
    out = rows * Hv * dv * e
    if case["op"] == "step":
        return {"bytes": tok + out + 2 * (B - case["pad"]) * Hv * dk * dv * 4, "flops": rows * Hv * 5 * dk * dv}
    states = len(_lens(case)) * Hv * dk * dv * 4
    if case["op"] == "fwd":
        return {"bytes": tok + out + states * (2 if case["state"] else 1), "flops": rows * Hv * 5 * dk * dv}
    return {"bytes": 2 * tok + out + (3 * states if case["state"] else 0), "flops": rows * Hv * 14 * dk * dv}
