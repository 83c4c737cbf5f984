"""Linear attention with a decay for each head and the norms with rotation where calls meet: captured into graphs and
replayed, two graphs on one workspace, on streams of their own, and over memory whose offsets pass 32 bits."""
import pytest

from gdr_testutil import check, gpu
from kda_testutil import say
from lad_testutil import make, reference, rotate, tol

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import chunked_gated_delta_amd as kda  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
NAMES = ("q", "k", "v", "w")


def lad(T=700, per_head=True, lens=None):
    d = gpu(make(1, T, 2, 4, 128, 64, BF16, "log", per_head=per_head, seed=1, states=len(lens) if lens else 1, layout="token"))
    d["cu"] = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda() if lens else None
    return d


def packed():
    return lad(900, False, [300, 0, 1, 599])


def rows():
    gen = torch.Generator().manual_seed(2)
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    d = dict(q=rn(2, 200, 4, 128), k=rn(2, 200, 2, 128), dq=rn(2, 200, 4, 128), dk=rn(2, 200, 2, 128))
    d = {n: x.to(BF16).cuda().transpose(1, 2) for n, x in d.items()}
    return dict(d, qw=torch.ones(128, device="cuda"), kw=1 + 0.1 * rn(128).cuda(), pos=torch.arange(200, dtype=torch.int32, device="cuda"),
                freq=torch.rand(64, generator=gen).cuda())


def step():
    d = gpu(make(5, 2, 2, 4, 64, 64, BF16, "log", per_head=True, seed=3, states=8))
    d["slots"] = torch.tensor([3, 0, -1, 3, 7], dtype=torch.int32, device="cuda")
    return d


ARGS = ("qw", "kw", "pos", "freq")
CALLS = {   # inputs; the call, which returns its results (updated states among them)
    "lad_chunk_fwd": (lad, lambda d, **s: kda.lad_chunk_fwd(*(d[n] for n in NAMES), d["S0"], log_decay=True, **s)),
    "lad_chunk_fwd packed": (packed, lambda d, **s: kda.lad_chunk_fwd(*(d[n] for n in NAMES), d["S0"], log_decay=True, cu_seqlens=d["cu"], **s)),
    "lad_chunk_bwd": (lad, lambda d, **s: kda.lad_chunk_bwd(*(d[n] for n in NAMES), d["dO"], d["S0"], d["dS_final"], log_decay=True, **s)),
    "lad_chunk_bwd packed": (packed, lambda d, **s: kda.lad_chunk_bwd(*(d[n] for n in NAMES), d["dO"], d["S0"], d["dS_final"], log_decay=True, cu_seqlens=d["cu"], **s)),
    "lad_decode": (step, lambda d, **s: (kda.lad_decode(*(d[n] for n in NAMES), d["S0"], d["slots"], log_decay=True, **s), d["S0"])),
    "qk_norm_rope_fwd": (rows, lambda d, **s: kda.qk_norm_rope_fwd(d["q"], d["k"], *(d[n] for n in ARGS), **s)),
    "qk_norm_rope_bwd": (rows, lambda d, **s: kda.qk_norm_rope_bwd(d["q"], d["k"], d["dq"], d["dk"], *(d[n] for n in ARGS), **s)),
}


def copies(d):
    out = {}
    for n, x in d.items():
        if x is not None:
            out[n] = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device=x.device)
            out[n].copy_(x)
        else:
            out[n] = None
    return out


def expected(name):
    make_inputs, call = CALLS[name]
    d = make_inputs()
    out = call(copies(d))
    torch.cuda.synchronize()
    return d, [x.clone() for x in out], call


def eager_work():
    x = torch.randn(1 << 20, device="cuda")
    return float((x - x.clone()).abs().sum())


@pytest.mark.parametrize("name", CALLS)
def test_captured(name):
    """Replays equal the eager call bit for bit, with the program's own work between them."""
    say(f"[case] {name} under graph capture")
    d, want, call = expected(name)
    t = copies(d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(copies(d))
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call(t)
    for i in range(4):
        for n, x in d.items():       # the inputs as they were: a step's states move on
            if x is not None:
                t[n].copy_(x)
        if name != "lad_decode":
            for x in out:
                x.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), (name, i)
        eager_work()


def test_two_graphs_on_one_workspace():
    """Graphs that are replayed one after another may share a workspace, which holds nothing between calls."""
    say("[case] two graphs on one workspace")
    a, b = lad(700), lad(1300)
    need = max(kda.lad_workspace_bytes(1, 2, 4, T, 128, 64, backward=True) for T in (700, 1300))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    calls = [lambda d=d: kda.lad_chunk_bwd(*(d[n] for n in NAMES), d["dO"], d["S0"], d["dS_final"], log_decay=True, workspace=ws) for d in (a, b)]
    want = [[x.clone() for x in c()] for c in calls]
    torch.cuda.synchronize()
    graphs = []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = c()
        graphs.append((g, out))
    for i in (0, 1, 1, 0, 0, 1):
        ws.fill_(0xAB)
        for x in graphs[i][1]:
            x.fill_(float("nan"))
        graphs[i][0].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(graphs[i][1], want[i])), i
        eager_work()


@pytest.mark.parametrize("name", CALLS)
def test_on_another_stream(name):
    """A call with `stream` while the current stream is busy, its results used there after a wait; memory that is dropped at once
    is not handed out before the call is done."""
    say(f"[case] {name} on another stream")
    d, want, call = expected(name)
    t = copies(d)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    x = torch.zeros(4096, 4096, dtype=BF16, device="cuda")
    with torch.cuda.stream(s):
        for _ in range(4):
            y = x @ x
    out = call(t, stream=s)
    kept = [o.data_ptr() for o in out]
    t = None
    fill = [torch.full((1 << 16,), 7.0, device="cuda") for _ in range(8)]     # takes what was dropped, if it may
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(out, want)), name
    assert len(fill) == 8 and len(kept) == len(out) and y.shape == x.shape


def test_two_streams_at_once():
    """The same call on two streams at the same time."""
    say("[case] two streams at once")
    d, want, call = expected("lad_chunk_bwd")
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [call(d, stream=s[i % 2]) for i in range(6)]
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, want))


def test_tokens_far_apart():
    """Tokens 2 MiB apart: rows lie up to 6 GB from the first."""
    say("[case] tokens far apart")
    T, D, H, gap = 3000, 64, 2, 1 << 20     # values between tokens
    buf = torch.zeros(T, gap, dtype=BF16, device="cuda")
    d = make(1, T, H, H, D, D, BF16, "log", per_head=True, seed=4, states=1)
    t = gpu(d)
    views = {}
    for i, n in enumerate(("q", "k", "v", "dO")):
        v = buf[:, i * H * D:(i + 1) * H * D].unflatten(-1, (H, D))[None].transpose(1, 2)
        v.copy_(t[n])
        views[n] = v
    out = buf[:, 8 * H * D:9 * H * D].unflatten(-1, (H, D))[None].transpose(1, 2)
    near = kda.lad_chunk_fwd(*(t[n] for n in NAMES), t["S0"], log_decay=True)
    far = kda.lad_chunk_fwd(views["q"], views["k"], views["v"], t["w"], t["S0"], log_decay=True)
    near_b = kda.lad_chunk_bwd(*(t[n] for n in NAMES), t["dO"], t["S0"], t["dS_final"], log_decay=True)
    far_b = kda.lad_chunk_bwd(views["q"], views["k"], views["v"], t["w"], views["dO"], t["S0"], t["dS_final"], log_decay=True)
    torch.cuda.synchronize()
    for a, b in zip(near + near_b, far + far_b):
        assert torch.equal(a, b)
    with pytest.raises(kda.KdaError, match="code -4"):      # an output between its inputs' rows
        kda.lad_chunk_fwd(views["q"], views["k"], views["v"], t["w"], out=out)
    del far, far_b
    y, _ = kda.qk_norm_rope_fwd(views["q"], None, None, None, torch.arange(T, dtype=torch.int32, device="cuda"), torch.ones(16, device="cuda"))
    z, _ = kda.qk_norm_rope_fwd(t["q"], None, None, None, torch.arange(T, dtype=torch.int32, device="cuda"), torch.ones(16, device="cuda"))
    assert torch.equal(y, z)


def test_states_far_into_a_pool():
    """A pool of 5 GB: slots behind 4 GB."""
    say("[case] states far into a pool")
    n, D = 80000, 128
    S = torch.zeros(n, 1, D, D, device="cuda")
    d = make(3, 1, 1, 1, D, D, F32, seed=5, states=3)
    t = gpu(d)
    slots = torch.tensor([n - 1, 66000, 5], dtype=torch.int32, device="cuda")
    S[slots.long()] = t["S0"]
    o = kda.lad_decode(*(t[n] for n in NAMES), S, slots)
    ro, rS = reference(d)
    check("o", o, ro, tol("o", F32))
    check("S", S[slots.long()], rS, tol("S", F32))
    assert int((S != 0).flatten(1).any(1).sum()) == 3


def test_long_sequence():
    """70000 tokens of one head whose state keeps everything: final state and last outputs against sums in 64 bits."""
    say("[case] a long sequence")
    T, D = 70000, 32
    gen = torch.Generator().manual_seed(6)
    q, k, v = (torch.randn(1, 1, T, D, generator=gen) for _ in range(3))
    w = torch.zeros(1)
    o, S = kda.lad_chunk_fwd(*(x.cuda() for x in (q, k, v, w)), log_decay=True)
    rS = k[0, 0].double().T @ v[0, 0].double()
    # a state of T products with sums of about sqrt(T): each chunk's sum is rounded to half a step of what has come together
    check("S_final", S[0, 0], rS, 4 * (T / 64) ** 0.5 * 2.0 ** -24)
    at = torch.arange(T - 40, T)
    ro = torch.stack([(q[0, 0, t].double() @ (k[0, 0, :t + 1].double().T @ v[0, 0, :t + 1].double())) for t in at.tolist()])
    check("o", o[0, 0, T - 40:], ro, 8 * (T / 64) ** 0.5 * 2.0 ** -24)


def test_rotation_of_many_tokens():
    """More tokens than one pass of workgroups, heads of two tensors, far positions."""
    say("[case] rotation of many tokens")
    T = 40000
    gen = torch.Generator().manual_seed(7)
    q, k = torch.randn(1, 3, T, 64, generator=gen), torch.randn(1, 1, T, 64, generator=gen)
    pos, freq = torch.arange(T, dtype=torch.int64) * 25, (1e6 ** (-torch.arange(0, 64, 2) / 64)).float()
    a, b = kda.qk_norm_rope_fwd(q.cuda(), k.cuda(), None, None, pos.cuda(), freq.cuda())
    check("q", a, rotate(q.double(), None, pos, freq), 32 * 2.0 ** -24)
    check("k", b, rotate(k.double(), None, pos, freq), 32 * 2.0 ** -24)
