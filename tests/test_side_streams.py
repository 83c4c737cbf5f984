"""Memory of calls on a stream that is not the current one.  The caching allocator may hand out a block as
soon as its tensor is dropped, to the stream that it was allocated on; so what a call makes is allocated on the stream
that writes it, and what it uses elsewhere is known to that stream.  Each test keeps one of the two streams busy
for some milliseconds, so that a block given away too early would be written in the wrong order."""
import pytest

from gdr_testutil import gpu, make
from kda_testutil import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import chunked_gated_delta_amd as kda  # noqa: E402

NAMES = ("q", "k", "v", "w", "beta")


def rule(dtype=torch.bfloat16):
    return gpu(make(1, 200, 2, 2, 128, 128, dtype, seed=1, states=1))


def channels():
    """The same with a gate per channel, for the per-channel rule."""
    d = rule()
    return dict(d, w=d["w"][..., None].repeat(1, 1, 1, 128))


def norms():
    gen = torch.Generator().manual_seed(2)
    rows = {n: torch.randn(900, 256, generator=gen).cuda() for n in ("x", "z", "residual", "ds", "dy")}
    return dict(rows, weight=torch.ones(256, device="cuda"), next_weight=torch.ones(256, device="cuda"))


NORM = ("weight", "z", "residual", "next_weight")
CALLS = {   # inputs; the call, which returns its results (updated states among them)
    "chunk_fwd": (channels, lambda d, s: kda.chunk_fwd(*(d[n] for n in NAMES), d["S0"], stream=s)),
    "chunk_fwd_noalloc": (channels, lambda d, s: kda.chunk_fwd_noalloc(*(d[n] for n in NAMES), d["S0"], stream=s)),
    "chunk_bwd": (channels, lambda d, s: kda.chunk_bwd(*(d[n] for n in NAMES), d["dO"], d["S0"], d["dS_final"], stream=s)),
    "decode": (channels, lambda d, s: (kda.decode(*(d[n] for n in NAMES), d["S0"], stream=s), d["S0"])),
    "gate_prefix": (channels, lambda d, s: kda.gate_prefix(d["w"], stream=s)),
    "gdr_chunk_fwd": (rule, lambda d, s: kda.gdr_chunk_fwd(*(d[n] for n in NAMES), d["S0"], stream=s)),
    "gdr_chunk_bwd": (rule, lambda d, s: kda.gdr_chunk_bwd(*(d[n] for n in NAMES), d["dO"], d["S0"], d["dS_final"], stream=s)),
    "gdr_decode": (rule, lambda d, s: (kda.gdr_decode(*(d[n] for n in NAMES), d["S0"], stream=s), d["S0"])),
    "norm_gate_fwd": (norms, lambda d, s: kda.norm_gate_fwd(d["x"], stream=s, **{n: d[n] for n in NORM})),
    "norm_gate_bwd": (norms, lambda d, s: kda.norm_gate_bwd(d["x"], d["ds"], d["dy"], stream=s, **{n: d[n] for n in NORM})),
}


def busy():
    """Some milliseconds of work on the current stream."""
    x = torch.zeros(8192, 8192, dtype=torch.bfloat16, device="cuda")
    for _ in range(4):
        x = x @ x


def copies(d):
    return {n: None if x is None else x.clone() for n, x in d.items()}


def same(got, ref):
    return all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, ref))


def reach(t):
    return t.untyped_storage().data_ptr(), t.untyped_storage().data_ptr() + t.untyped_storage().nbytes()


@pytest.mark.parametrize("name", CALLS)
def test_memory_still_in_use_on_the_current_stream(name):
    """What the call makes does not lie where the current stream has yet to write and read."""
    make_inputs, call = CALLS[name]
    say(f"[case] {name} on a side stream, temporaries of the current one dropped")
    d = make_inputs()
    ref = [x.clone() for x in call(copies(d), None)]
    torch.cuda.synchronize()
    side, e = torch.cuda.Stream(), copies(d)
    torch.cuda.synchronize()
    busy()
    temps = [torch.empty_like(x) for _ in range(3) for x in ref] + [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (1 << 20, 1 << 23)]
    seen = []
    for t in temps:
        t.fill_(1)
        seen.append(t.clone())
    places = [reach(t) for t in temps]
    del t, temps   # free for the current stream, whose work on them has not begun
    got = call(e, side)
    for x in got:
        if not any(x is y for y in e.values()):
            lo, hi = reach(x)
            assert all(hi <= a or b <= lo for a, b in places), "a result lies in memory that the current stream still uses"
    torch.cuda.synchronize()
    assert same(got, ref) and all((x == 1).all() for x in seen)


@pytest.mark.parametrize("name", CALLS)
def test_inputs_dropped_while_the_side_stream_is_busy(name):
    make_inputs, call = CALLS[name]
    say(f"[case] {name} on a busy side stream, inputs dropped")
    d = make_inputs()
    ref = [x.clone() for x in call(copies(d), None)]
    side, e = torch.cuda.Stream(), copies(d)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        busy()
    got = call(e, side)
    sizes = [x.numel() * x.element_size() for x in e.values() if x is not None]
    del e
    for n in sizes:
        for _ in range(3):   # would take the inputs' places
            torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert same(got, ref)


@pytest.mark.parametrize("name", CALLS)
def test_results_dropped_while_the_current_stream_reads_them(name):
    make_inputs, call = CALLS[name]
    say(f"[case] {name} on a side stream, results read late")
    d = make_inputs()
    ref = [x.clone() for x in call(copies(d), None)]
    f = {n: None if x is None else -x for n, x in d.items()}   # other values: the second call's results differ
    side, e = torch.cuda.Stream(), copies(d)
    torch.cuda.synchronize()
    got = call(e, side)
    torch.cuda.current_stream().wait_stream(side)
    busy()
    seen = [x.clone() for x in got]
    del got, e
    call(f, side)   # would take the places of the first call's results
    torch.cuda.synchronize()
    assert same(seen, ref)


@pytest.mark.parametrize("name", ["decode", "gdr_decode", "norm_gate_fwd"])
def test_a_stream_of_its_own_device(name):
    """A stream of another device is refused before anything is allocated or launched."""
    make_inputs, call = CALLS[name]

    class Elsewhere:
        device, cuda_stream = torch.device("cuda", 99), 0

    with pytest.raises(ValueError, match="stream is on"):
        call(make_inputs(), Elsewhere())


@pytest.mark.parametrize("name", ["chunk_fwd", "chunk_bwd", "gdr_chunk_fwd", "gdr_chunk_bwd", "norm_gate_bwd"])
def test_captured_on_a_stream_that_forks_off(name):
    """A call on a second stream inside a captured graph, replayed with eager work between."""
    make_inputs, call = CALLS[name]
    say(f"[case] {name} on a forked stream of a graph")
    d = make_inputs()
    ref = [x.clone() for x in call(d, None)]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        out = call(d, side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(4):
        for x in out:
            x.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, ref)
        assert same(call(d, None), ref)   # the program's own calls between replays
