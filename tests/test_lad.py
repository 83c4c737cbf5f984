"""Linear attention with a decay for each head on the GPU (chunked forward, gradients, recurrent step) against the
token recurrence in 64 bits."""
import math

import pytest

from gdr_testutil import check, gate_args, gpu, half
from kda_testutil import say
from lad_testutil import F32 as F32_TOL
from lad_testutil import SPLIT, make, reference, tol

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from chunked_gated_delta_amd import lad_chunk_bwd, lad_chunk_fwd, lad_decode  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
NAMES = ("q", "k", "v", "w")
GRADS = ("dq", "dk", "dv", "dw", "dS0")


def offsets(lens):
    return torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda() if lens is not None else None


def run_fwd(d, lens=None, gate="bounded", scale=1.0, **kw):
    t = gpu(d)
    r = lad_chunk_fwd(*(t[n] for n in NAMES), t["S0"], cu_seqlens=offsets(lens), scale=scale, **gate_args(gate), **kw)
    torch.cuda.synchronize()
    return r


def run_bwd(d, lens=None, gate="bounded", scale=1.0, **kw):
    t = gpu(d)
    r = lad_chunk_bwd(*(t[n] for n in NAMES), t["dO"], t["S0"], t["dS_final"], cu_seqlens=offsets(lens), scale=scale, **gate_args(gate), **kw)
    torch.cuda.synchronize()
    return r


UNIFORM = [  # B, T, Hk, Hv, dk, dv, gate, per head, states, layout
    (1, 1, 1, 1, 32, 32, "bounded", False, 0, "head"),
    (2, 15, 1, 1, 32, 64, "softplus", False, 1, "token"),
    (1, 64, 2, 4, 64, 32, "bounded", True, 0, "token"),
    (1, 65, 1, 3, 128, 128, "log", False, 1, "head"),
    (3, 63, 2, 2, 64, 128, "softplus", True, 1, "token"),
    (2, 130, 2, 4, 128, 64, "bounded", False, 1, "token"),
    (1, 333, 3, 3, 128, 128, "log", True, 0, "head"),
    (1, 517, 1, 2, 32, 128, "log", False, 1, "token"),
    (1, 700, 1, 1, 128, 32, "softplus", False, 1, "head"),
    (2, 300, 1, 2, 64, 64, "log", True, 1, "token"),
]
PACKED = [  # lens, tokens behind the last sequence, Hk, Hv, dk, dv, gate, per head, states
    ([64, 0, 1, 63, 65, 130], 0, 2, 4, 128, 128, "bounded", False, True),
    ([0, 0], 5, 1, 1, 32, 32, "softplus", False, True),
    ([1, 1, 1, 127], 9, 1, 2, 64, 32, "log", True, False),
    ([200], 70, 1, 1, 32, 64, "bounded", False, True),
    ([0, 530, 3, 0, 257, 256], 11, 1, 2, 128, 64, "log", True, True),
    ([600, 513], 0, 1, 1, 64, 128, "softplus", False, False),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", UNIFORM, ids=str)
def test_forward(case, dtype):
    B, T, Hk, Hv, dk, dv, gate, per_head, states, layout = case
    say(f"[case] lad forward {case} {dtype}")
    d = make(B, T, Hk, Hv, dk, dv, dtype, gate, per_head, seed=1, states=B * states, layout=layout)
    o, S = run_fwd(d, gate=gate, scale=dk ** -0.5)
    ro, rS = reference(d, gate=gate, scale=dk ** -0.5)
    assert o.dtype == dtype and o.stride() == d["v"].stride()
    check("o", o, ro, tol("o", dtype))
    check("S_final", S, rS, tol("S", dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", PACKED, ids=str)
def test_forward_packed(case, dtype):
    lens, behind, Hk, Hv, dk, dv, gate, per_head, states = case
    say(f"[case] lad packed forward {case} {dtype}")
    T = sum(lens)
    d = make(1, T + behind, Hk, Hv, dk, dv, dtype, gate, per_head, seed=2, states=len(lens) if states else 0, layout="token")
    for n in NAMES[:3 if per_head else 4]:   # nothing behind the last sequence is read
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
    B, T, Hk, Hv, dk, dv, gate, per_head, states, layout = case
    say(f"[case] lad backward {case} {dtype}")
    d = make(B, T, Hk, Hv, dk, dv, dtype, gate, per_head, seed=3, states=B * states, layout=layout)
    got = run_bwd(d, gate=gate, scale=dk ** -0.5)
    _, _, ref = reference(d, gate=gate, scale=dk ** -0.5, grads=True)
    for n, x in zip(GRADS, got):
        if n in ref:
            assert x.dtype == (F32 if n == "dS0" or (n == "dw" and per_head) else dtype)
            check(n, x, ref[n], tol(n, dtype, per_head), more=1e-6 if T == 1 and n == "dw" else 0.0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", PACKED, ids=str)
def test_backward_packed(case, dtype):
    lens, behind, Hk, Hv, dk, dv, gate, per_head, states = case
    say(f"[case] lad packed backward {case} {dtype}")
    T = sum(lens)
    d = make(1, T + behind, Hk, Hv, dk, dv, dtype, gate, per_head, seed=4, states=len(lens) if states else 0)
    rows = NAMES[:3 if per_head else 4] + ("dO",)
    for n in rows:
        d[n][:, :, T:] = float("nan")
    got = run_bwd(d, lens, gate, 0.5)
    if T == 0:   # no token: the states' adjoints pass through
        assert torch.equal(got[4].cpu(), d["dS_final"])
        return
    for n in rows:
        d[n] = d[n][:, :, :T]
    _, _, ref = reference(d, lens, gate, 0.5, grads=True)
    for n, x in zip(GRADS, got):
        if n in ref:
            check(n, x if n == "dS0" or x.dim() == 1 else x[:, :, :T], ref[n], tol(n, dtype, per_head))


@pytest.mark.parametrize("want_dw,want_dS0,dSf", [(False, False, True), (False, True, False), (True, False, True), (True, True, False), (True, False, False)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [90, 700])
def test_backward_in_part(T, dtype, want_dw, want_dS0, dSf):
    """What is not wanted is left out, and the rest is what it was."""
    say(f"[case] lad backward in part {T} {dtype} {want_dw} {want_dS0} {dSf}")
    d = make(1, T, 1, 2, 64, 32, dtype, seed=5, states=1)
    if not dSf:
        d["dS_final"] = None
    got = run_bwd(d, want_dw=want_dw, want_dS0=want_dS0)
    _, _, ref = reference(d, grads=True)
    for n, x in zip(GRADS, got):
        if (n == "dw" and not want_dw) or (n == "dS0" and not want_dS0):
            assert x is None
        else:
            check(n, x, ref[n], tol(n, dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_resets(dtype):
    """Log-decays of -infinity and of the type's lowest value forget the state exactly; one of 0 keeps everything."""
    say(f"[case] lad resets {dtype}")
    d = make(1, 600, 1, 2, 64, 64, dtype, "log", seed=5, states=1)
    d["w"][:, :, 20] = -math.inf
    d["w"][:, :, 90] = torch.finfo(dtype).min
    d["w"][:, 0, 550] = -math.inf
    d["w"][:, :, 100:120] = 0.0
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


@pytest.mark.parametrize("g", [0.0, -math.inf])
def test_heads_that_keep_or_forget_everything(g):
    say(f"[case] lad decay {g}")
    d = make(1, 140, 2, 2, 32, 32, F32, "log", per_head=True, seed=6, states=1)
    d["w"][0] = g
    o, S = run_fwd(d, gate="log")
    ro, rS = reference(d, gate="log")
    check("o", o, ro, tol("o", F32))
    check("S_final", S, rS, tol("S", F32))


@pytest.mark.parametrize("n", [2, 511, 700])
def test_many_sequences(n):
    say(f"[case] lad {n} sequences")
    lens = torch.randint(0, 4, (n,), generator=torch.Generator().manual_seed(n)).tolist()
    lens[n // 2] = 130
    d = make(1, sum(lens), 1, 1, 32, 32, F32, seed=16, states=n)
    o, S = run_fwd(d, lens)
    ro, rS, ref = reference(d, lens, grads=True)
    check("o", o, ro, tol("o", F32))
    check("S_final", S, rS, tol("S", F32))
    for m, x in zip(GRADS, run_bwd(d, lens)):
        check(m, x, ref[m], tol(m, F32))


@pytest.mark.parametrize("case", [(1, 150, 2, 4, 128, 128, "bounded"), (2, 2, 1, 4, 32, 64, "softplus"), (3, 77, 2, 2, 64, 32, "log"), (1, 600, 1, 1, 128, 128, "log")])
def test_bf16_results_are_rounded_once(case):
    """The results' error is their own rounding's: what lies before it is off by the planes' 2^-17 alone."""
    B, T, Hk, Hv, dk, dv, gate = case
    say(f"[case] lad rounded once {case}")
    d = make(B, T, Hk, Hv, dk, dv, BF16, gate, seed=15, states=B)
    ro, _, ref = reference(d, gate=gate, grads=True)
    o, _ = run_fwd(d, gate=gate)
    for n, got, r in [("o", o, ro)] + [(n, x, ref[n]) for n, x in zip(GRADS, run_bwd(d, gate=gate)) if n != "dS0"]:
        r = r.detach().double()
        own = float((r.to(BF16).double() - r).norm()) / float(r.norm())
        check(n, got, r, own + SPLIT * (32 if n == "dw" else 1))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [130, 500, 1100])
def test_states_keep_fp32s_accuracy(T, dtype):
    """Final states and dS0 of 3, 8 and 18 chunks: sums in fp32 of two parts a chunk, each off by half a step of what has come
    together, 2 sqrt(36) half steps = 7.2e-7 at most; two bf16 planes in place of three are off by 2e-6 and more."""
    say(f"[case] lad states {T} {dtype}")
    d = make(1, T, 2, 2, 128, 128, dtype, "log", per_head=True, seed=8, states=1)
    _, S = run_fwd(d, gate="log")
    _, rS, ref = reference(d, gate="log", grads=True)
    check("S_final", S, rS, 7.2e-7)
    check("dS0", run_bwd(d, gate="log")[4], ref["dS0"], 7.2e-7)


def test_state_in_place_and_chained():
    """S_final may be S0; two calls from whole chunks equal one call to rounding."""
    say("[case] lad chained")
    d = make(1, 1280, 2, 2, 128, 128, BF16, seed=6, states=1)
    t = gpu(d)
    args = [t[n] for n in NAMES]
    o, S = lad_chunk_fwd(*args, t["S0"])
    St = t["S0"].clone()
    o1, _ = lad_chunk_fwd(*(x[:, :, :640] for x in args), St, S_final=St)
    o2, S2 = lad_chunk_fwd(*(x[:, :, 640:] for x in args), St, S_final=St)
    torch.cuda.synchronize()
    assert S2 is St
    check("o", torch.cat([o1, o2], 2), o.double().cpu(), 2 * tol("o", BF16))   # both are rounded
    check("S", St, S.double().cpu(), 2 * F32_TOL)


def test_strided_views():
    """Slices of one fused projection, a broadcast key head and a strided output."""
    say("[case] lad views")
    T, H, D = 100, 2, 64
    gen = torch.Generator().manual_seed(7)
    x = torch.randn(1, T, 3 * H * D, generator=gen).to(BF16).cuda()
    q, v = (x[..., i * H * D:(i + 1) * H * D].unflatten(-1, (H, D)).transpose(1, 2) for i in (0, 2))
    k = (0.1 * x[..., H * D:H * D + D])[:, None].expand(1, H, T, D)
    w = torch.randn(1, T, 1, generator=gen).to(BF16).cuda().transpose(1, 2).expand(1, H, T)
    dO = torch.randn(1, H, T, D, generator=gen).to(BF16).cuda()
    out = torch.full((1, T, H, 2 * D), 5.0, dtype=BF16, device="cuda")
    o, S = lad_chunk_fwd(q, k, v, w, out=out[..., :D].transpose(1, 2))
    got = lad_chunk_bwd(q, k, v, w, dO)
    d = dict(q=q.cpu(), k=k.cpu(), v=v.cpu(), w=w.cpu(), dO=dO.cpu(), S0=None, dS_final=None)
    ro, rS, ref = reference(d, grads=True)
    check("o", o, ro, tol("o", BF16))
    check("S", S, rS, tol("S", BF16))
    assert (out[..., D:] == 5).all()
    for n, g in zip(GRADS[:4], got):
        check(n, g, ref[n], tol(n, BF16))


def test_offsets_out_of_order_stay_inside():
    """Offsets out of order or range give undefined values; nothing outside the tensors is read or written."""
    say("[case] lad offsets out of order")
    T, H, D = 300, 2, 32
    d = make(1, T, H, H, D, D, BF16, seed=9)
    t = gpu(d)
    pad = torch.full((1, H, T + 64, D), 3.0, dtype=BF16, device="cuda")
    for cu in ([0, 200, 100, 300], [250, 10, 400, -5], [-100, 50, 1 << 30, 60], [300, 0, 0, 0]):
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        lad_chunk_fwd(*(t[n] for n in NAMES), cu_seqlens=c, out=pad[:, :, :T])
        lad_chunk_bwd(*(t[n] for n in NAMES), t["dO"], cu_seqlens=c)
        torch.cuda.synchronize()
        assert (pad[:, :, T:] == 3).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_nan_stays_in_its_sequence(dtype):
    """A NaN and an infinity in the tokens of one sequence leave the others as they are, forwards and in the gradients."""
    say(f"[case] lad with a NaN {dtype}")
    lens = [70, 300, 129]
    d = make(1, sum(lens), 1, 2, 64, 64, dtype, seed=19, states=3)
    clean = run_fwd(d, lens) + run_bwd(d, lens)
    for n, i in (("k", 75), ("v", 90), ("q", 200), ("w", 150)):
        d[n][:, :, i] = float("nan") if n != "v" else float("inf")
    got = run_fwd(d, lens) + run_bwd(d, lens)
    for x, y in zip(got, clean):
        if x.shape[0] == 3:
            assert torch.equal(x[[0, 2]], y[[0, 2]])
        else:
            assert torch.equal(x[:, :, :70], y[:, :, :70]) and torch.equal(x[:, :, 370:], y[:, :, 370:])
    assert not torch.isfinite(got[0][:, :, 70:370]).all()


def test_runs_are_equal():
    """The same call gives the same bits."""
    say("[case] lad runs")
    d = make(2, 900, 2, 4, 64, 64, BF16, seed=10, states=2)
    a, b = run_fwd(d) + run_bwd(d), run_fwd(d) + run_bwd(d)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_gradients_against_differences():
    """The gradients of a loss agree with central differences of the forward along random directions (fp32)."""
    say("[case] lad differences")
    d = make(1, 130, 1, 2, 32, 32, F32, "log", seed=11, states=1)
    got = dict(zip(GRADS, run_bwd(d, gate="log")))

    def loss(e):
        o, S = run_fwd(e, gate="log")
        return float((o.double().cpu() * d["dO"].double()).sum() + (S.double().cpu() * d["dS_final"].double()).sum())

    gen = torch.Generator().manual_seed(12)
    h = 2.0 ** -7
    for n in NAMES + ("S0",):
        u = torch.randn(d[n].shape, generator=gen)
        u = u / u.norm() * (0.05 if n == "w" else 1.0)
        lo, hi = dict(d), dict(d)
        lo[n], hi[n] = d[n] - h * u, d[n] + h * u
        by_diff = (loss(hi) - loss(lo)) / (2 * h)
        by_grad = float((got["d" + n].double().cpu() * u.double()).sum())
        size = float(got["d" + n].double().cpu().norm()) * float(u.double().norm())
        # the loss sums 8000 products of fp32 results: off by 1e-5 at most, over 2 h; the third derivative by h^2
        say(f"   d{n}: {by_grad:.6f} by gradient, {by_diff:.6f} by differences")
        assert abs(by_diff - by_grad) <= 2e-3 * size + 1e-5 / h


STEPS = [  # B, slots, T, Hk, Hv, dk, dv, gate, per head
    (1, 1, 1, 1, 1, 32, 32, "bounded", False),
    (5, 9, 1, 2, 4, 128, 128, "softplus", False),
    (3, 3, 4, 1, 3, 64, 128, "log", True),
    (7, 8, 2, 2, 2, 128, 32, "bounded", True),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", STEPS, ids=str)
def test_decode(case, dtype):
    """Rows with a state of the pool, a padding row, and states that no row names."""
    B, slots, T, Hk, Hv, dk, dv, gate, per_head = case
    say(f"[case] lad decode {case} {dtype}")
    d = make(B, T, Hk, Hv, dk, dv, dtype, gate, per_head, seed=13, states=slots, layout="token")
    at = torch.randperm(slots, generator=torch.Generator().manual_seed(1))[:B].to(torch.int32)
    if B > 2:
        at[1] = -1
    t = gpu(d)
    S = t["S0"].clone()
    o = lad_decode(*(t[n] for n in NAMES), S, at.cuda(), scale=0.5, **gate_args(gate))
    torch.cuda.synchronize()
    live = [b for b in range(B) if at[b] >= 0]
    e = {n: (x if x is None or x.dim() == 1 else x[live]) for n, x in d.items() if n not in ("S0", "dS_final")}
    e["S0"] = d["S0"][at[live].long()]
    ro, rS = reference(e, gate=gate, scale=0.5)
    check("o", o[live], ro, half(dtype) + F32_TOL)
    check("S", S.cpu()[at[live].long()], rS, F32_TOL)
    others = [i for i in range(slots) if i not in at[live].tolist()]
    assert torch.equal(S.cpu()[others], d["S0"][others])
    if B > 2:
        assert (o[1] == 0).all()


def test_decode_same_slot_and_every_row():
    """Rows with one slot are successive tokens; without slots row b has state b."""
    say("[case] lad decode, one slot twice")
    d = make(6, 2, 1, 2, 64, 64, F32, seed=14, states=4)
    t = gpu(d)
    S = t["S0"].clone()
    at = torch.tensor([2, 0, 2, 7, 2, 0], dtype=torch.int32)
    o = lad_decode(*(t[n] for n in NAMES), S, at.cuda())
    for s in (0, 2):
        rows = [b for b in range(6) if at[b] == s]
        e = {n: torch.cat([d[n][b:b + 1] for b in rows], 2) for n in NAMES + ("dO",)}
        ro, rS = reference(dict(e, S0=d["S0"][s:s + 1], dS_final=None))
        check("o", torch.cat([o[b:b + 1] for b in rows], 2), ro, F32_TOL)
        check("S", S[s:s + 1], rS, F32_TOL)
    assert (o[3] == 0).all() and torch.equal(S[[1, 3]].cpu(), d["S0"][[1, 3]])
    S = t["S0"].clone()
    o = lad_decode(*(t[n][:4] for n in NAMES), S)
    ro, rS = reference({n: (x[:4] if x is not None else None) for n, x in d.items()})
    check("o", o, ro, F32_TOL)
    check("S", S, rS, F32_TOL)


def test_decode_continues_the_chunked_form():
    """A prompt through the chunked form, then tokens one by one, equal the whole sequence's chunked form."""
    say("[case] lad prompt, then tokens")
    d = make(2, 140, 2, 4, 128, 64, F32, "log", per_head=True, seed=17, states=2)
    t = gpu(d)
    o, S = lad_chunk_fwd(*(t[n] for n in NAMES), t["S0"], log_decay=True)
    cut = lambda a, b: [t[n][:, :, a:b] for n in NAMES[:3]] + [t["w"]]  # noqa: E731
    outs, (first, St) = [], lad_chunk_fwd(*cut(0, 130), t["S0"], log_decay=True)
    outs.append(first)
    for i in range(130, 140):
        outs.append(lad_decode(*cut(i, i + 1), St, log_decay=True))
    check("o", torch.cat(outs, 2), o.double().cpu(), 2 * F32_TOL)
    check("S", St, S.double().cpu(), 2 * F32_TOL)


def test_no_tokens():
    say("[case] lad without tokens")
    for T in (0,):
        d = make(2, T, 1, 1, 32, 32, BF16, per_head=True, seed=18, states=2)
        o, S = run_fwd(d)
        assert o.shape == (2, 1, 0, 32) and torch.equal(S.cpu(), d["S0"])
        got = run_bwd(d)
        assert torch.equal(got[4].cpu(), d["dS_final"]) and (got[3] == 0).all()
