"""The head-gated delta rule on the GPU (chunked forward, gradients, recurrent step) against the token
recurrence in 64 bits."""
import math

import pytest

from gdr_testutil import SPLIT, check, gate_args, gpu, make, reference, tol
from kda_testutil import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from chunked_gated_delta_amd import gdr_chunk_bwd, gdr_chunk_fwd, gdr_decode  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
NAMES = ("q", "k", "v", "w", "beta")
GRADS = ("dq", "dk", "dv", "dw", "dbeta", "dS0")


def offsets(lens):
    return torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda() if lens is not None else None


def run_fwd(d, lens=None, gate="bounded", scale=1.0, **kw):
    t = gpu(d)
    r = gdr_chunk_fwd(*(t[n] for n in NAMES), t["S0"], cu_seqlens=offsets(lens), scale=scale, **gate_args(gate), **kw)
    torch.cuda.synchronize()
    return r


def run_bwd(d, lens=None, gate="bounded", scale=1.0, **kw):
    t = gpu(d)
    r = gdr_chunk_bwd(*(t[n] for n in NAMES), t["dO"], t["S0"], t["dS_final"], cu_seqlens=offsets(lens), scale=scale, **gate_args(gate), **kw)
    torch.cuda.synchronize()
    return r


UNIFORM = [  # B, T, Hk, Hv, dk, dv, gate, states, layout
    (1, 1, 1, 1, 32, 32, "bounded", 0, "head"),
    (2, 15, 1, 1, 32, 64, "softplus", 1, "token"),
    (1, 64, 2, 4, 64, 32, "bounded", 0, "token"),
    (1, 65, 1, 3, 128, 128, "log", 1, "head"),
    (3, 63, 2, 2, 64, 128, "softplus", 1, "token"),
    (2, 130, 2, 4, 128, 64, "bounded", 1, "token"),
    (1, 333, 3, 3, 128, 128, "softplus", 0, "head"),
    (1, 517, 1, 2, 32, 128, "log", 1, "token"),
]
PACKED = [  # lens, tokens behind the last sequence, Hk, Hv, dk, dv, gate, states
    ([64, 0, 1, 63, 65, 130], 0, 2, 4, 128, 128, "bounded", True),
    ([0, 0], 5, 1, 1, 32, 32, "softplus", True),
    ([1, 1, 1, 127], 9, 1, 2, 64, 32, "log", False),
    ([200], 70, 1, 1, 32, 64, "bounded", True),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", UNIFORM, ids=str)
def test_forward(case, dtype):
    B, T, Hk, Hv, dk, dv, gate, states, layout = case
    say(f"[case] gdr forward {case} {dtype}")
    d = make(B, T, Hk, Hv, dk, dv, dtype, gate, seed=1, states=B * states, layout=layout)
    o, S = run_fwd(d, gate=gate, scale=dk ** -0.5)
    ro, rS = reference(d, gate=gate, scale=dk ** -0.5)
    assert o.dtype == dtype and o.stride() == d["v"].stride()
    check("o", o, ro, tol("o", dtype))
    check("S_final", S, rS, tol("S", dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", PACKED, ids=str)
def test_forward_packed(case, dtype):
    lens, behind, Hk, Hv, dk, dv, gate, states = case
    say(f"[case] gdr packed forward {case} {dtype}")
    T = sum(lens)
    d = make(1, T + behind, Hk, Hv, dk, dv, dtype, gate, seed=2, states=len(lens) if states else 0, layout="token")
    for n in NAMES:   # nothing behind the last sequence is read
        d[n][:, :, T:] = float("nan")
    out = torch.full((1, Hv, T + behind, dv), 7.0, dtype=dtype, device="cuda")
    o, S = run_fwd(d, lens, gate, 0.25, out=out)
    ro, rS = reference(d, lens, gate, 0.25)
    check("o", o[:, :, :T], ro, tol("o", dtype))
    check("S_final", S, rS, tol("S", dtype))
    assert (o[:, :, T:] == 7).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", UNIFORM, ids=str)
def test_backward(case, dtype):
    B, T, Hk, Hv, dk, dv, gate, states, layout = case
    say(f"[case] gdr backward {case} {dtype}")
    d = make(B, T, Hk, Hv, dk, dv, dtype, gate, seed=3, states=B * states, layout=layout)
    got = run_bwd(d, gate=gate, scale=dk ** -0.5)
    _, _, ref = reference(d, gate=gate, scale=dk ** -0.5, grads=True)
    for n, x in zip(GRADS, got):
        if n in ref:
            assert x.dtype == (F32 if n == "dS0" else dtype)
            check(n, x, ref[n], tol(n, dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", PACKED, ids=str)
def test_backward_packed(case, dtype):
    lens, behind, Hk, Hv, dk, dv, gate, states = case
    say(f"[case] gdr packed backward {case} {dtype}")
    T = sum(lens)
    d = make(1, T + behind, Hk, Hv, dk, dv, dtype, gate, seed=4, states=len(lens) if states else 0)
    for n in NAMES + ("dO",):
        d[n][:, :, T:] = float("nan")
    got = run_bwd(d, lens, gate, 0.5)
    if T == 0:   # no token: the states' adjoints pass through
        assert torch.equal(got[5].cpu(), d["dS_final"])
        return
    for n in NAMES + ("dO",):
        d[n] = d[n][:, :, :T]
    _, _, ref = reference(d, lens, gate, 0.5, grads=True)
    for n, x in zip(GRADS, got):
        if n in ref:
            check(n, x if n == "dS0" else x[:, :, :T], ref[n], tol(n, dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_resets_and_zero_rates(dtype):
    """Log-decays of -infinity and of the type's lowest value forget the state exactly; beta 0 writes nothing
    and still has a gradient; a log-decay of 0 keeps everything."""
    say(f"[case] gdr resets {dtype}")
    d = make(1, 150, 1, 2, 64, 64, dtype, "log", seed=5, states=1)
    d["w"][:, :, 20] = -math.inf
    d["w"][:, :, 90] = torch.finfo(dtype).min
    d["w"][:, :, 100:120] = 0.0
    d["beta"][:, :, 30:40] = 0.0
    d["beta"][:, 1, 64:130] = 0.0
    o, S = run_fwd(d, gate="log")
    ro, rS = reference(d, gate="log")
    check("o", o, ro, tol("o", dtype))
    check("S_final", S, rS, tol("S", dtype))
    got = run_bwd(d, gate="log")
    e = {n: x.clone() if x is not None else None for n, x in d.items()}
    e["w"].clamp_(min=-1e4)     # the same decays, with a finite derivative
    _, _, ref = reference(e, gate="log", grads=True)
    for n, x in zip(GRADS, got):
        check(n, x, ref[n], tol(n, dtype))


@pytest.mark.parametrize("n", [2, 511, 512, 513, 700])
def test_many_sequences(n):
    """Batches on both sides of the number of sequences that are taken longest first; equal lengths among them."""
    say(f"[case] gdr {n} sequences")
    lens = torch.randint(0, 4, (n,), generator=torch.Generator().manual_seed(n)).tolist()
    lens[n // 2] = 130
    d = make(1, sum(lens), 1, 1, 32, 32, F32, seed=16, states=n)
    o, S = run_fwd(d, lens)
    ro, rS, ref = reference(d, lens, grads=True)
    check("o", o, ro, tol("o", F32))
    check("S_final", S, rS, tol("S", F32))
    for m, x in zip(GRADS, run_bwd(d, lens)):
        check(m, x, ref[m], tol(m, F32))


@pytest.mark.parametrize("case", [(1, 150, 2, 4, 128, 128, "bounded"), (2, 2, 1, 4, 32, 64, "softplus"), (3, 77, 2, 2, 64, 32, "log")])
def test_bf16_results_are_rounded_once(case):
    """The results' error is their own rounding's: what lies before it is off by the planes' 2^-17 alone."""
    B, T, Hk, Hv, dk, dv, gate = case
    say(f"[case] gdr rounded once {case}")
    d = make(B, T, Hk, Hv, dk, dv, BF16, gate, seed=15, states=B)
    ro, _, ref = reference(d, gate=gate, grads=True)
    o, _ = run_fwd(d, gate=gate)
    for n, got, r in [("o", o, ro)] + [(n, x, ref[n]) for n, x in zip(GRADS, run_bwd(d, gate=gate)) if n != "dS0"]:
        r = r.detach().double()
        own = float((r.to(BF16).double() - r).norm()) / float(r.norm())
        check(n, got, r, own + SPLIT * (8 if n == "dw" else 1))


def test_state_in_place_and_chained():
    """S_final may be S0; two calls from whole chunks equal one call to rounding."""
    say("[case] gdr chained")
    d = make(1, 256, 2, 2, 128, 128, BF16, seed=6, states=1)
    t = gpu(d)
    args = [t[n] for n in NAMES]
    o, S = gdr_chunk_fwd(*args, t["S0"])
    St = t["S0"].clone()
    o1, _ = gdr_chunk_fwd(*(x[:, :, :128] for x in args), St, S_final=St)
    o2, S2 = gdr_chunk_fwd(*(x[:, :, 128:] for x in args), St, S_final=St)
    torch.cuda.synchronize()
    assert S2 is St
    check("o", torch.cat([o1, o2], 2), o.double().cpu(), 2 * tol("o", BF16))   # both are rounded
    check("S", St, S.double().cpu(), tol("S", BF16))


def test_strided_views():
    """Slices of one fused projection, a broadcast key head and a strided output."""
    say("[case] gdr views")
    T, H, D = 100, 2, 64
    gen = torch.Generator().manual_seed(7)
    x = torch.randn(1, T, 3 * H * D, generator=gen).to(BF16)
    q, k, v = (0.2 * x[..., :H * D].unflatten(-1, (H, D)), None, x[..., 2 * H * D:].unflatten(-1, (H, D)))
    buf = torch.cat([q.flatten(2), x[..., H * D:]], -1).cuda()
    qg, vg = (buf[..., i * H * D:(i + 1) * H * D].unflatten(-1, (H, D)).transpose(1, 2) for i in (0, 2))
    k1 = (0.1 * torch.randn(1, 1, T, D, generator=gen)).to(BF16)
    d = make(1, T, H, H, D, D, BF16, seed=8)
    kg = k1.cuda().expand(1, H, T, D)
    w, beta = d["w"].cuda(), d["beta"].cuda()
    big = torch.full((1, T, H, 2 * D), 3.0, dtype=BF16, device="cuda")
    o, S = gdr_chunk_fwd(qg, kg, vg, w, beta, out=big[..., :D].transpose(1, 2))
    e = dict(d, q=qg.cpu(), k=k1.expand(1, H, T, D), v=vg.cpu())
    ro, rS = reference(e)
    check("o", o, ro, tol("o", BF16))
    check("S", S, rS, tol("S", BF16))
    assert (big[..., D:] == 3).all()
    got = gdr_chunk_bwd(qg, kg, vg, w, beta, d["dO"].cuda())
    _, _, ref = reference(e, grads=True)
    for n, y in zip(GRADS, got[:5]):
        check(n, y, ref[n], tol(n, BF16))


def test_nothing_crosses_sequences():
    """NaN and infinities in one packed sequence reach no other, nor earlier chunks of their own."""
    say("[case] gdr isolation")
    lens = [100, 70, 90]
    d = make(1, 260, 1, 1, 32, 32, BF16, seed=9)
    clean = run_fwd(d, lens)
    cb = run_bwd(d, lens)
    for n in ("q", "k", "v"):
        d[n][:, :, 165:170] = float("nan") if n == "q" else math.inf
    o, S = run_fwd(d, lens)
    b = run_bwd(d, lens)
    for x, y in [(o, clean[0])] + list(zip(b[:5], cb[:5])):
        assert torch.equal(x[:, :, :100], y[:, :, :100]) and torch.equal(x[:, :, 170:], y[:, :, 170:])
    assert torch.equal(o[:, :, 100:164], clean[0][:, :, 100:164])
    assert torch.equal(S[[0, 2]], clean[1][[0, 2]])


def test_offsets_out_of_order_are_harmless():
    """Offsets outside the tokens, or falling, are clamped: no access out of range, the call returns."""
    say("[case] gdr bad offsets")
    d = gpu(make(1, 200, 1, 1, 32, 32, BF16, seed=10))
    guard = torch.full((3, 1, 200, 32), 5.0, dtype=BF16, device="cuda")
    cu = torch.tensor([-70, 300, 100, 2 ** 31 - 1, -2 ** 31, 200], dtype=torch.int32, device="cuda")
    gdr_chunk_fwd(*(d[n] for n in NAMES), cu_seqlens=cu, out=guard[1:2])
    gdr_chunk_bwd(*(d[n] for n in NAMES), d["dO"], cu_seqlens=cu)
    torch.cuda.synchronize()
    assert (guard[0] == 5).all() and (guard[2] == 5).all()


# ------------------------------------------------------------------------------------------------- recurrent step


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", [(1, 1, 1, 1, 32, 32, "bounded"), (5, 1, 2, 4, 128, 128, "softplus"), (3, 4, 1, 3, 64, 128, "log"),
                                  (70, 2, 1, 1, 128, 32, "bounded"), (4, 1, 4, 4, 32, 64, "log")], ids=str)
def test_step(case, dtype):
    """Rows of a pool by slot, padding among them; the states of no row stay as they were."""
    B, T, Hk, Hv, dk, dv, gate = case
    say(f"[case] gdr step {case} {dtype}")
    d = make(B, T, Hk, Hv, dk, dv, dtype, gate, seed=11, states=B + 2, layout="token")
    order = torch.randperm(B + 2, generator=torch.Generator().manual_seed(1))[:B].to(torch.int32)
    if B > 2:
        order[1], order[B - 1] = -1, B + 2
    t = gpu(d)
    S = t["S0"].clone()
    o = gdr_decode(*(t[n] for n in NAMES), S, order.cuda(), scale=0.3, **gate_args(gate))
    torch.cuda.synchronize()
    live = ((order >= 0) & (order < B + 2)).nonzero()[:, 0]
    e = {n: d[n][live] if d[n] is not None and n not in ("S0", "dS_final") else None for n in d}
    e["S0"] = d["S0"][order[live].long()]
    ro, rS = reference(e, gate=gate, scale=0.3)
    check("o", o[live.cuda()], ro, tol("o", dtype))
    check("S", S[order[live].long().cuda()], rS, tol("S", F32))
    rest = torch.ones(B + 2, dtype=torch.bool)
    rest[order[live].long()] = False
    assert torch.equal(S.cpu()[rest], d["S0"][rest])
    if B > 2:
        assert (o[[1, B - 1]] == 0).all()


def test_step_rows_of_one_slot_are_its_tokens():
    say("[case] gdr step, one slot in several rows")
    d = make(6, 2, 1, 2, 64, 64, F32, seed=12, states=3)
    order = torch.tensor([2, 0, 2, -1, 2, 0], dtype=torch.int32)
    t = gpu(d)
    S = t["S0"].clone()
    o = gdr_decode(*(t[n] for n in NAMES), S, order.cuda())
    torch.cuda.synchronize()
    for slot, rows in ((2, [0, 2, 4]), (0, [1, 5])):
        e = {n: torch.cat([d[n][r:r + 1] for r in rows], 2) for n in NAMES}
        ro, rS = reference(dict(e, S0=d["S0"][slot:slot + 1], dS_final=None))
        check("o", torch.cat([o[r:r + 1] for r in rows], 2), ro, tol("o", F32))
        check("S", S[slot:slot + 1], rS, tol("S", F32))
    assert torch.equal(S[1].cpu(), d["S0"][1]) and (o[3] == 0).all()


def test_step_in_a_pool_past_32_bits():
    """70000 states of 64 KiB: the last one's bytes lie behind 2^32."""
    say("[case] gdr step, large pool")
    d = make(2, 1, 1, 1, 128, 128, BF16, seed=13, states=2)
    t = gpu(d)
    S = torch.zeros(70000, 1, 128, 128, device="cuda")
    S[69999], S[3] = t["S0"][0], t["S0"][1]
    o = gdr_decode(*(t[n] for n in NAMES), S, torch.tensor([69999, 3], dtype=torch.int32, device="cuda"))
    ro, rS = reference(d)
    check("o", o, ro, tol("o", BF16))
    check("S", S[[69999, 3]], rS, tol("S", F32))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prefill_then_answer(dtype):
    """Packed prompts, their states scattered to a pool, four steps: the whole sequences' chunked outputs."""
    from chunked_gated_delta_amd import norm_gate_fwd
    say(f"[case] gdr prefill, steps and the gated norm {dtype}")
    lens, extra = [70, 1, 129], 4
    full = [make(1, n + extra, 1, 2, 128, 64, dtype, "softplus", seed=20 + i, layout="token") for i, n in enumerate(lens)]
    kw = dict(g_min=-math.inf, scale=128 ** -0.5)
    packed = {n: torch.cat([f[n][:, :, :m] for f, m in zip(full, lens)], 2).cuda() for n in NAMES}
    o, S = gdr_chunk_fwd(*(packed[n] for n in NAMES), cu_seqlens=offsets(lens), **kw)
    pool = torch.zeros(5, 2, 128, 64, device="cuda")
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    pool[slots.long()] = S
    steps = []
    for j in range(extra):
        tok = {n: torch.cat([f[n][:, :, m + j:m + j + 1] for f, m in zip(full, lens)], 0).cuda() for n in NAMES}
        steps.append(gdr_decode(*(tok[n] for n in NAMES), pool, slots, **kw))
    weight = torch.linspace(0.5, 1.5, 64, device="cuda")
    z = torch.linspace(-2, 2, 64, device="cuda").to(dtype).expand(1, 2, 3 + 1, 64)
    at = 0
    for i, (f, m) in enumerate(zip(full, lens)):
        ro, rS = reference(f, gate="softplus", scale=128 ** -0.5)
        check("o", torch.cat([o[:, :, at:at + m]] + [s[i:i + 1] for s in steps], 2), ro, tol("o", dtype))
        check("S", pool[slots[i].long()][None], rS, tol("S", dtype))
        at += m
        y, _ = norm_gate_fwd(torch.cat([s[i:i + 1] for s in steps], 2), weight, z)
        zz = z.double().cpu()
        r = ro[:, :, m:]
        r = r / torch.sqrt((r * r).mean(-1, keepdim=True) + 1e-6) * weight.double().cpu() * zz * torch.sigmoid(zz)
        check("norm of o", y, r, 2 * tol("o", dtype))


# --------------------------------------------------------------------------------------------- streams and graphs


def test_other_stream_and_two_at_once():
    """Calls on side streams, two at a time, equal the calls on the current stream bit for bit."""
    say("[case] gdr streams")
    d = [gpu(make(1, 700, 2, 4, 128, 128, BF16, seed=30 + i, states=1)) for i in range(2)]
    f = lambda t, **kw: gdr_chunk_fwd(*(t[n] for n in NAMES), t["S0"], **kw)  # noqa: E731
    b = lambda t, **kw: gdr_chunk_bwd(*(t[n] for n in NAMES), t["dO"], t["S0"], t["dS_final"], **kw)  # noqa: E731
    ref = [[x.clone() for x in f(t) + b(t)] for t in d]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in d]
    got = [f(t, stream=s) + b(t, stream=s) for t, s in zip(d, streams)]
    torch.cuda.synchronize()
    for r, g in zip(ref, got):
        assert all(torch.equal(x, y) for x, y in zip(r, g))


def test_graph_replays():
    """Forward, backward and step captured into one graph with their own workspaces, replayed with eager
    work between."""
    say("[case] gdr graph")
    d = gpu(make(1, 300, 1, 2, 128, 128, BF16, seed=40, states=1))
    args = [d[n] for n in NAMES]
    pool = d["S0"].clone()
    one = [x[:, :, :1] for x in args]
    slots = torch.zeros(1, dtype=torch.int32, device="cuda")

    def work():
        o, S = gdr_chunk_fwd(*args, d["S0"])
        g = gdr_chunk_bwd(*args, d["dO"], d["S0"], d["dS_final"])
        pool.copy_(S)
        return (o, S) + g + (gdr_decode(*one, pool, slots), pool)

    ref = [x.clone() for x in work()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for _ in range(4):
        for x in out:
            x.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, ref))
        eager = work()          # the program's own calls between replays
        assert float(torch.randn(1 << 20, device="cuda").sum()) != 0 and all(torch.equal(x, y) for x, y in zip(eager, ref))


def test_gradient_by_differences():
    """fp32: the gradients along random directions against central differences of the forward.  A step of 2^-6
    leaves the third-order term, h^2 / 6 of third derivatives of order 10: 4e-4, and rounding, 1e-6 / h: 6e-5."""
    say("[case] gdr differences")
    d = make(1, 80, 1, 2, 32, 32, F32, "softplus", seed=50, states=1)
    got = dict(zip(GRADS, run_bwd(d, gate="softplus", scale=0.5)))
    gen = torch.Generator().manual_seed(1)

    def loss(e):
        o, S = run_fwd(e, gate="softplus", scale=0.5)
        return float((o.double().cpu() * d["dO"].double()).sum() + (S.double().cpu() * d["dS_final"].double()).sum())

    h = 2.0 ** -6
    for n in NAMES + ("S0",):
        u = torch.randn(d[n].shape, generator=gen)
        u /= u.norm()
        lo, hi = (loss(dict(d, **{n: d[n] + s * h * u})) for s in (-1, 1))
        want = float((got["d" + n].double().cpu() * u.double()).sum())
        size = float(got["d" + n].double().norm())
        say(f"   {n}: {want:.6f} by the gradient, {(hi - lo) / 2 / h:.6f} by differences")
        assert abs((hi - lo) / 2 / h - want) <= 5e-4 * size
