"""Cases of the head-gated delta rule (chunked forward, its gradients, the recurrent step on a pool of
states) and of the norms around a block, in a plain form and through this package's entry points.

`own` False: elementary torch operations in 32 bits (in 64 for the cumulative log-decays and for the
gate's gradient, sums of cancelling terms), rounded once at the end.  `own` True: the calls a user makes.

The head-gated delta rule, per sequence and value head, with a state S (dk x dv) and one log-decay per token:
    S <- e^{g_t} S;  f_t = v_t - S^T k_t;  S <- S + beta_t k_t f_t^T;  o_t = scale S^T q_t
with g = g_min sigmoid(w), -softplus(w) or w itself; value head h reads query and key head h / (Hv / Hk).

The norms around a block, per row of D values:
    n = x / rms(x) * weight;  h = n * act(z);  s = residual + alpha h;  y = s / rms(s) * next_weight
where every part but one of the two norms may be absent.
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
        dict(name="fwd one prompt of 130", op="fwd", B=1, lens="", T=130, Hk=4, Hv=4, dk=128, dv=128, dtype="bf16", gate="bounded",
             layout="token", state=True),
        # a serving step's prompts packed one behind another: an empty one, one token, chunk borders, shared key heads
        dict(name="fwd packed prompts", op="fwd", B=1, lens="517,0,1,64,1300,63,65,2000,89", T=4099, Hk=8, Hv=16, dk=128, dv=128,
             dtype="bf16", gate="softplus", layout="fused", state=True),
        # one document of this repository's headline length and heads
        dict(name="fwd 64K tokens", op="fwd", B=1, lens="", T=65536, Hk=16, Hv=16, dk=128, dv=128, dtype="bf16", gate="bounded",
             layout="head", state=False),
        # fp32 inputs, an odd length and unequal head sizes
        dict(name="fwd fp32 1001", op="fwd", B=2, lens="", T=1001, Hk=4, Hv=8, dk=64, dv=32, dtype="f32", gate="log", layout="head",
             state=True),
        # the gradients of a training step at this repository's 4096-token batch
        dict(name="bwd 2x4096", op="bwd", B=2, lens="", T=4096, Hk=16, Hv=16, dk=128, dv=128, dtype="bf16", gate="bounded",
             layout="token", state=False),
        # fp32 gradients of packed documents with shared key heads and entering states
        dict(name="bwd fp32 packed", op="bwd", B=1, lens="300,1,0,447,64", T=812, Hk=2, Hv=4, dk=64, dv=128, dtype="f32",
             gate="softplus", layout="token", state=True),
        # one sequence that answers token by token
        dict(name="step 1 sequence", op="step", B=1, slots=4, pad=0, T=1, Hk=4, Hv=8, dk=128, dv=128, dtype="bf16", gate="bounded"),
        # a serving batch of 512 rows, some of them padding, over a larger pool
        dict(name="step 512 sequences", op="step", B=512, slots=528, pad=7, T=1, Hk=8, Hv=16, dk=128, dv=128, dtype="bf16",
             gate="bounded"),
        # the gated norm of the heads' outputs while answering: few rows
        dict(name="norm heads 3 tokens", op="norm", dir="fwd", form="heads", N=3, H=16, D=128, dtype="bf16", act="silu", wdtype="f32"),
        # residual and both norms around a block, a ragged number of rows
        dict(name="norm block 8191x4096", op="norm", dir="fwd", form="block", N=8191, H=1, D=4096, dtype="bf16", act="sigmoid",
             wdtype="bf16"),
        # gradients of the heads' gated norm at the 4096-token batch
        dict(name="norm heads bwd 2x4096", op="norm", dir="bwd", form="heads", N=8192, H=16, D=128, dtype="bf16", act="sigmoid",
             wdtype="f32"),
        # gradients of residual add and pre-norm, an odd row size, fp32
        dict(name="norm add bwd fp32", op="norm", dir="bwd", form="add", N=1500, H=1, D=1111, dtype="f32", act="none", wdtype="f32"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "step", "norm", "norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        form = rng.choice(["heads", "block", "add"])
        D = rng.choice([32, 64, 128, 256]) if form == "heads" else _spread(rng, 100, 8192)
        H = rng.choice([1, 4, 16]) if form == "heads" else 1
        N = _spread(rng, 1, max(2, (1 << 24) // (D * H)))
        return dict(op="norm", dir=rng.choice(["fwd", "bwd"]), form=form, N=N, H=H, D=D, dtype=dtype,
                    act=rng.choice(["silu", "sigmoid", "none"]), wdtype=rng.choice([dtype, "f32"]))
    Hk, grp = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4])
    case = dict(op=op, Hk=Hk, Hv=Hk * grp, dk=rng.choice([32, 64, 128]), dv=rng.choice([32, 64, 128]), dtype=dtype,
                gate=rng.choice(["bounded", "softplus", "log"]))
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


def prepare(case, seed):
    """The inputs, on the GPU, from the seed alone."""
    dev = _device()
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    dt = _TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    st = {"case": case}
    if case["op"] == "norm":
        N, H, D = case["N"], case["H"], case["D"]
        wt = _TYPES[case["wdtype"]]
        view = lambda x: x.to(dt).view(1, N, H, D).transpose(1, 2)  # noqa: E731  [1, H, N, D], a token's heads side by side
        st["x"] = view(normal(N, H, D) * torch.exp(0.5 * normal(N, 1, 1)))
        form = case["form"]
        st["weight"] = (1 + 0.1 * normal(D)).to(wt) if form != "add" else None
        st["z"] = view(1.5 * normal(N, H, D)) if form != "add" and case["act"] != "none" else None
        st["residual"] = view(2 * normal(N, H, D)) if form != "heads" else None
        st["next_weight"] = (1 + 0.1 * normal(D)).to(wt) if form != "heads" else None
        st["alpha"] = 1.0 if form == "heads" else 0.75
        if case["dir"] == "bwd":
            st["ds"] = view(normal(N, H, D))
            st["dy"] = view(normal(N, H, D)) if form != "heads" else None
        return st
    B, T, Hk, Hv, dk, dv = (case[n] for n in ("B", "T", "Hk", "Hv", "dk", "dv"))
    layout = case.get("layout", "head")
    q, k, v = _unit(normal(B, T, Hk, dk)).to(dt), _unit(normal(B, T, Hk, dk)).to(dt), normal(B, T, Hv, dv).to(dt)
    if layout == "fused":     # one projection's output, its columns divided into queries, keys and values
        x = torch.cat([q.flatten(2), k.flatten(2), v.flatten(2)], dim=-1)
        a, b = Hk * dk, 2 * Hk * dk
        q, k, v = x[..., :a].unflatten(-1, (Hk, dk)), x[..., a:b].unflatten(-1, (Hk, dk)), x[..., b:].unflatten(-1, (Hv, dv))
    q, k, v = (x.transpose(1, 2) for x in (q, k, v))
    w = 2 * normal(B, T, Hv)
    w = (torch.nn.functional.logsigmoid(w + 2) if case["gate"] == "log" else w).to(dt).transpose(1, 2)
    beta = torch.sigmoid(normal(B, T, Hv)).to(dt).transpose(1, 2)
    if layout == "head":
        q, k, v, w, beta = (x.contiguous() for x in (q, k, v, w, beta))
    st.update(q=q, k=k, v=v, w=w, beta=beta, scale=dk ** -0.5)
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
        st["dO"] = dO.contiguous() if layout == "head" else dO
        st["dS_final"] = 0.3 * normal(len(lens), Hv, dk, dv) if case["state"] else None
    return st


# ------------------------------------------------------------------------------------------------------------ plain forms


def _gate(w, gate):
    """The log-decay and its derivative by w."""
    if gate == "log":
        return w, torch.ones_like(w)
    s = 1 / (1 + torch.exp(-w))
    if gate == "bounded":
        return G_MIN * s, G_MIN * s * (1 - s)
    return -(torch.clamp_min(w, 0) + torch.log1p(torch.exp(-w.abs()))), -s


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


def _inverse(A):
    """(I + A)^{-1} of strictly lower triangular A (64 x 64, so A^64 = 0): (I - A)(I + A^2)(I + A^4) ... (I + A^32)."""
    eye = torch.eye(CHUNK, device=A.device, dtype=A.dtype)
    inv = eye - A
    for _ in range(5):
        A = A @ A
        inv = inv @ (eye + A)
    return inv


def _chunks(st):
    """What both directions of the chunk form start with, per sequence, value head and chunk of 64 tokens."""
    c = st["case"]
    grp = c["Hv"] // c["Hk"]
    p = {}
    for n in ("q", "k", "v"):
        x = _pad(st[n], st).float().unflatten(2, (-1, CHUNK))
        p[n] = x.repeat_interleave(grp, 1) if n != "v" else x
    w, b = _pad(st["w"], st).double(), _pad(st["beta"], st).float()
    g, p["dgate"] = _gate(w, c["gate"])
    if st["cu_seqlens"] is None:
        live = (torch.arange(w.shape[2], device=w.device) < st["t_max"]).expand_as(w)
    else:
        cu = st["cu_seqlens"]
        live = (torch.arange(w.shape[2], device=w.device)[None, None] < (cu[1:] - cu[:-1])[:, None, None]).expand_as(w)
    g = torch.where(live, g, 0.0).unflatten(2, (-1, CHUNK))
    p["beta"] = b.unflatten(2, (-1, CHUNK))[..., None]
    G = g.cumsum(-1)
    p["D"] = torch.exp((G[..., :, None] - G[..., None, :]).tril()).float().tril()
    p["gam"], p["eta"], p["last"] = G.exp().float()[..., None], (G[..., -1:] - G).exp().float()[..., None], G[..., -1].exp().float()[..., None, None]
    p["KK"] = (p["k"] @ p["k"].transpose(-1, -2) * p["D"]).tril(-1)
    p["QK"] = (p["q"] @ p["k"].transpose(-1, -2) * p["D"]) * st["scale"]
    inv = _inverse(p["KK"] * p["beta"].transpose(-1, -2))
    W, U0 = inv @ (p["gam"] * p["k"]), inv @ p["v"]
    Keta = (p["eta"] * p["k"]).transpose(-1, -2)
    n, H, nc = U0.shape[:3]
    S = st["S0"].clone() if st["S0"] is not None else U0.new_zeros(n, H, c["dk"], c["dv"])
    states, fs = [], []
    for i in range(nc):
        F = U0[:, :, i] - W[:, :, i] @ S
        states.append(S)
        fs.append(F)
        S = p["last"][:, :, i] * S + Keta[:, :, i] @ (p["beta"][:, :, i] * F)
    p["S"], p["F"], p["S_final"] = torch.stack(states, 2), torch.stack(fs, 2), S
    return p


def _plain_fwd(st):
    p = _chunks(st)
    o = st["scale"] * p["gam"] * (p["q"] @ p["S"]) + p["QK"] @ (p["beta"] * p["F"])
    return _unpad(o.flatten(2, 3), st).to(st["v"].dtype), p["S_final"]


def _plain_bwd(st):
    c = st["case"]
    p = _chunks(st)
    T_ = lambda x: x.transpose(-1, -2)  # noqa: E731
    scale, k, q, F, S, beta, gam, eta = st["scale"], p["k"], p["q"], p["F"], p["S"], p["beta"], p["gam"], p["eta"]
    dO = scale * _pad(st["dO"], st).float().unflatten(2, (-1, CHUNK))
    inv = T_(_inverse(p["KK"] * beta))
    X0, dS0 = T_(p["QK"] / scale) @ dO, T_(gam * q) @ dO
    Kgam, Keta = T_(gam * k), eta * k
    dS = st["dS_final"].clone() if st["dS_final"] is not None else torch.zeros_like(S[:, :, 0])
    nc = S.shape[2]
    dSs, dUs = [None] * nc, [None] * nc
    for i in reversed(range(nc)):
        dU = inv[:, :, i] @ (X0[:, :, i] + Keta[:, :, i] @ dS)
        dSs[i], dUs[i] = dS, dU
        dS = p["last"][:, :, i] * dS + dS0[:, :, i] - Kgam[:, :, i] @ (beta[:, :, i] * dU)
    dSn, dU = torch.stack(dSs, 2), torch.stack(dUs, 2)
    U, dE = beta * F, beta * dU
    dP = dO @ T_(U) * p["D"]
    dA = -(dE @ T_(U) * p["D"]).tril(-1)
    dq_ = gam * (dO @ T_(S)) + dP @ k
    dk_row = -gam * (dE @ T_(S)) + dA @ k
    dk_col = eta * (U @ T_(dSn)) + T_(dA) @ k + T_(dP) @ q
    # the log-decay's gradient: cancelling terms, summed in 64 bits
    dG = (q.double() * dq_ + k.double() * dk_row - k.double() * dk_col).sum(-1)
    dG[..., -1] += (k.double() * eta * (U @ T_(dSn))).sum((-1, -2)) + (p["last"].double() * S * dSn).sum((-1, -2))
    dg = dG.flip(-1).cumsum(-1).flip(-1).flatten(2, 3)
    n, _, _, C, dk = dq_.shape
    heads = lambda x: x.view(n, c["Hk"], -1, nc, C, dk).sum(2)  # noqa: E731  value heads that share a key head
    out = [heads(dq_), heads(dk_row + dk_col), dE, dg * p["dgate"], (dU * F).sum(-1)]
    out = [_unpad((x.flatten(2, 3) if i != 3 else x).to(st["q"].dtype), st) for i, x in enumerate(out)]
    return tuple(out) + ((dS,) if st["S0"] is not None else ())


def _plain_step(st):
    c = st["case"]
    grp = c["Hv"] // c["Hk"]
    at = st["slots"].long()
    keep = (at >= 0)[:, None, None, None]
    S = st["S"][at.clamp_min(0)]
    q, k, v = st["q"].float().repeat_interleave(grp, 1), st["k"].float().repeat_interleave(grp, 1), st["v"].float()
    a, beta = torch.exp(_gate(st["w"].float(), c["gate"])[0]), st["beta"].float()
    outs = []
    for t in range(c["T"]):
        S = a[:, :, t, None, None] * S
        f = v[:, :, t] - (S * k[:, :, t, :, None]).sum(-2)
        S = S + k[:, :, t, :, None] * (beta[:, :, t, None] * f)[:, :, None]
        outs.append(st["scale"] * (S * q[:, :, t, :, None]).sum(-2))
    # padding rows go to a row behind the pool, which is dropped
    pool = torch.cat([st["S"], torch.zeros_like(st["S"][:1])])
    pool[torch.where(at >= 0, at, st["S"].shape[0])] = S
    st["S"].copy_(pool[:-1])
    return torch.where(keep, torch.stack(outs, 2), 0.0).to(st["v"].dtype), st["S"]


def _act(z, act):
    """act(z) and its derivative."""
    s = 1 / (1 + torch.exp(-z))
    return (s, s * (1 - s)) if act == "sigmoid" else (z * s, s * (1 + z * (1 - s)))


def _norm(st, f):
    """The norms around a block in type f: (s, y), or the gradients."""
    c = st["case"]
    up = lambda n: st[n].to(f) if st.get(n) is not None else None  # noqa: E731
    x, w, z, res, w2, alpha = up("x"), up("weight"), up("z"), up("residual"), up("next_weight"), st["alpha"]
    n, r = x, None
    if w is not None:
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        n = x * r * w
    a, da = _act(z, c["act"]) if z is not None else (1.0, None)
    s = alpha * n * a + (res if res is not None else 0.0)
    r2 = torch.rsqrt(s.square().mean(-1, keepdim=True) + EPS) if w2 is not None else None
    if c["dir"] == "fwd":
        return (s,) if w2 is None else (s, s * r2 * w2)
    ds, dy = up("ds"), up("dy")
    dw = dw2 = dz = None
    if w2 is not None:
        sh, t = s * r2, dy * w2
        dw2 = (dy * sh).sum((0, 1, 2))
        ds = ds + r2 * (t - sh * (t * sh).mean(-1, keepdim=True))
    dn = alpha * ds * a
    if z is not None:
        dz = alpha * ds * n * da
    dx = dn
    if w is not None:
        xh, t = x * r, dn * w
        dw = (dn * xh).sum((0, 1, 2))
        dx = r * (t - xh * (t * xh).mean(-1, keepdim=True))
    return dx, dw, dz, ds if res is not None else None, dw2


def _norm_types(st, out):
    """The outputs in the types that they come in: a row's values as x, weights' gradients as the weights."""
    dt = st["x"].dtype
    if st["case"]["dir"] == "fwd":
        return tuple(v.to(dt) for v in out)
    wt = (st["weight"] if st["weight"] is not None else st["next_weight"]).dtype
    return tuple(None if v is None else v.to(wt if i in (1, 4) else dt) for i, v in enumerate(out))


# ------------------------------------------------------------------------------------------------------------------- run


def _gate_args(case):
    return {"bounded": dict(g_min=G_MIN), "softplus": dict(g_min=-math.inf), "log": dict(log_decay=True)}[case["gate"]]


def run(state):
    """One pass through the operator."""
    st, c = state, state["case"]
    if not own:
        if c["op"] == "norm":
            return _norm_types(st, _norm(st, torch.float32))
        return {"fwd": _plain_fwd, "bwd": _plain_bwd, "step": _plain_step}[c["op"]](st)
    import chunked_gated_delta_amd as kda
    if c["op"] == "norm":
        args = dict(weight=st["weight"], z=st["z"], act=c["act"], residual=st["residual"], alpha=st["alpha"], next_weight=st["next_weight"], eps=EPS)
        if c["dir"] == "fwd":
            s, y = kda.norm_gate_fwd(st["x"], **args)
            return (s,) if y is None else (s, y)
        return kda.norm_gate_bwd(st["x"], st["ds"], st["dy"], **args)
    args = [st[n] for n in ("q", "k", "v", "w", "beta")]
    kw = dict(scale=st["scale"], **_gate_args(c))
    if c["op"] == "step":
        return kda.gdr_decode(*args, st["S"], st["slots"], **kw), st["S"]
    if c["op"] == "fwd":
        return kda.gdr_chunk_fwd(*args, st["S0"], cu_seqlens=st["cu_seqlens"], **kw)
    out = kda.gdr_chunk_bwd(*args, st["dO"], st["S0"], st["dS_final"], cu_seqlens=st["cu_seqlens"], want_dS0=st["S0"] is not None, **kw)
    return out if st["S0"] is not None else out[:5]


# ------------------------------------------------------------------------------------------- the definition, in 64 bits


def exact(case, seed):
    """run()'s answer from the token recurrence (and its adjoint) in 64 bits."""
    st = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(st)
    return _exact_step(st) if case["op"] == "step" else _exact_rule(st)


def _exact_gate(w, gate):
    w = w.double()
    if gate == "bounded":
        return G_MIN * torch.sigmoid(w), G_MIN * torch.sigmoid(w) * torch.sigmoid(-w)
    if gate == "softplus":
        return torch.nn.functional.logsigmoid(-w), -torch.sigmoid(w)
    return w, torch.ones_like(w)


def _exact_rule(st):
    c, grp = st["case"], st["case"]["Hv"] // st["case"]["Hk"]
    ends = st["cu_seqlens"].tolist() if st["cu_seqlens"] is not None else None
    g, dgate = _exact_gate(st["w"], c["gate"])
    q, k = (st[n].double().repeat_interleave(grp, 1) for n in ("q", "k"))
    v, beta, bwd = st["v"].double(), st["beta"].double(), c["op"] == "bwd"
    o = torch.zeros_like(v)
    dq, dk, dv, dg, db = (torch.zeros_like(x) for x in (q, k, v, g, beta))
    dO = st["dO"].double() if bwd else None
    finals, starts = [], []
    spans = [(slice(None), 0, c["T"], slice(None))] if ends is None else [(slice(0, 1), a, b, slice(i, i + 1)) for i, (a, b) in enumerate(zip(ends, ends[1:]))]
    for rows, a, b, at in spans:
        n = c["B"] if ends is None else 1
        S = st["S0"][at].double() if st["S0"] is not None else v.new_zeros(n, c["Hv"], c["dk"], c["dv"])
        kept = []
        for t in range(a, b):
            kt, decay = k[rows, :, t, :, None], g[rows, :, t, None, None].exp()
            old = decay * S
            f = v[rows, :, t] - (old * kt).sum(-2)
            S = old + kt * (beta[rows, :, t, None] * f)[:, :, None]
            o[rows, :, t] = st["scale"] * (S * q[rows, :, t, :, None]).sum(-2)
            if bwd:
                kept.append((old, f, S))
        finals.append(S)
        if not bwd:
            continue
        dS = st["dS_final"][at].double() if st["dS_final"] is not None else torch.zeros_like(S)
        for t in reversed(range(a, b)):
            old, f, S = kept.pop()
            kt, bt, do = k[rows, :, t, :, None], beta[rows, :, t, None], st["scale"] * dO[rows, :, t, None]
            dS = dS + q[rows, :, t, :, None] * do
            dq[rows, :, t] = (S * do).sum(-1)
            u, du = (bt * f)[:, :, None], (dS * kt).sum(-2)
            df = bt * du
            db[rows, :, t], dv[rows, :, t] = (du * f).sum(-1), df
            dold = dS - kt * df[:, :, None]
            dk[rows, :, t] = (dS * u).sum(-1) - (old * df[:, :, None]).sum(-1)
            dg[rows, :, t] = (dold * old).sum((-1, -2))
            dS = g[rows, :, t, None, None].exp() * dold
        starts.append(dS)
    if not bwd:
        return o, torch.cat(finals)
    shared = lambda x: x.unflatten(1, (c["Hk"], grp)).sum(2)  # noqa: E731
    out = (shared(dq), shared(dk), dv, dg * dgate, db)
    return out + ((torch.cat(starts),) if st["S0"] is not None else ())


def _exact_step(st):
    c, grp = st["case"], st["case"]["Hv"] // st["case"]["Hk"]
    o, pool = torch.zeros_like(st["v"], dtype=torch.float64), st["S"]
    at = st["slots"].long()
    rows = (at >= 0).nonzero()[:, 0]
    S = pool[at[rows]].double()
    q, k = (st[n][rows].double().repeat_interleave(grp, 1) for n in ("q", "k"))
    v, beta, g = st["v"][rows].double(), st["beta"][rows].double(), _exact_gate(st["w"][rows], c["gate"])[0]
    for t in range(c["T"]):
        S = S * g[:, :, t, None, None].exp()
        f = v[:, :, t] - (k[:, :, t, None] @ S)[:, :, 0]
        S = S + k[:, :, t, :, None] * (beta[:, :, t, None] * f)[:, :, None]
        o[rows, :, t] = st["scale"] * (q[:, :, t, None] @ S)[:, :, 0]
    pool = pool.double()
    pool[at[rows]] = S
    return o, pool


def _exact_norm(st):
    """By automatic differentiation of the definition."""
    c = st["case"]
    leaf = {n: st[n].double().requires_grad_() for n in ("x", "weight", "z", "residual", "next_weight") if st.get(n) is not None}
    rms = lambda t: (t.pow(2).sum(-1, keepdim=True) / c["D"] + EPS).sqrt()  # noqa: E731
    h = leaf["x"]
    if "weight" in leaf:
        h = h / rms(h) * leaf["weight"]
    if "z" in leaf:
        h = h * (torch.sigmoid(leaf["z"]) if c["act"] == "sigmoid" else leaf["z"] * torch.sigmoid(leaf["z"]))
    s = st["alpha"] * h
    if "residual" in leaf:
        s = s + leaf["residual"]
    outs = [s] + ([s / rms(s) * leaf["next_weight"]] if "next_weight" in leaf else [])
    if c["dir"] == "fwd":
        return tuple(x.detach() for x in outs)
    names = [n for n in ("x", "weight", "z", "residual", "next_weight") if n in leaf]
    got = dict(zip(names, torch.autograd.grad(outs, [leaf[n] for n in names], [st[n].double() for n in ("ds", "dy")[:len(outs)]])))
    return tuple(got.get(n) for n in ("x", "weight", "z", "residual", "next_weight"))


# ------------------------------------------------------------------------------------------------------------------ work


def work(case):
    """Bytes read and written once each, and the recurrence's multiplications and additions."""
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        n, D = case["N"] * case["H"] * case["D"], case["D"]
        form, we = case["form"], 2 if case["wdtype"] == "bf16" else 4
        gate = form != "add" and case["act"] != "none"
        ins = 1 + gate + (form != "heads")
        norms = (form != "add") + (form != "heads")
        if case["dir"] == "fwd":
            return {"bytes": n * e * (ins + 1 + (form != "heads")) + norms * D * we, "flops": n * (4 * norms + 5 * gate + 2)}
        return {"bytes": n * e * (2 * ins + 1 + (form != "heads")) + 2 * norms * D * we, "flops": n * (12 * norms + 10 * gate + 4)}
    Hk, Hv, dk, dv, B, T = (case[n] for n in ("Hk", "Hv", "dk", "dv", "B", "T"))
    rows = (B - case["pad"] if case["op"] == "step" else B) * T
    tok = rows * (2 * Hk * dk + Hv * dv + 2 * Hv) * e      # q, k, v, w, beta
    out = rows * Hv * dv * e
    if case["op"] == "step":
        return {"bytes": tok + out + 2 * (B - case["pad"]) * Hv * dk * dv * 4, "flops": rows * Hv * 7 * dk * dv}
    states = len(_lens(case)) * Hv * dk * dv * 4
    if case["op"] == "fwd":
        return {"bytes": tok + out + states * (2 if case["state"] else 1), "flops": rows * Hv * 7 * dk * dv}
    return {"bytes": 2 * tok + out + (3 * states if case["state"] else 0), "flops": rows * Hv * 19 * dk * dv}
