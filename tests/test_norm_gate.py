"""The norms around a block (gated norm of heads, residual add with the next norm, both) on the GPU against
64 bits: every part present or absent, odd row sizes, strided rows, gradients.

Tolerances: outputs and rows' gradients are computed in fp32 and rounded once: half a step of their type, and for
fp32 (and beside it) 64 half steps of fp32, the sums over a row (up to 16384 values, added in a tree of at most 32
values a thread and 9 levels) and four products.  dx through the first norm is the difference r t - r x/rms(x) c of
terms that are each off by those 64 half steps of their own size |r t|; in a row of one value the two cancel
to eps / (x^2 + eps) of that size (1 - x^2 / (x^2 + eps)), 1e-7 at x = 3, below a single rounding of either
term, so the terms' size is what the error is measured by.  Weights' gradients are sums over rows with random signs: 64
half steps of fp32 for the same reason, and their type's half step."""
import pytest

from gdr_testutil import check, half, norms
from kda_testutil import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from chunked_gated_delta_amd import norm_gate_bwd, norm_gate_fwd  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
T32 = 64 * half(F32)
FORMS = {"heads": ("weight", "z"), "norm": ("weight",), "add": ("residual", "next_weight"), "both": ("weight", "residual", "next_weight"),
         "block": ("weight", "z", "residual", "next_weight"), "gate": ("z", "next_weight"), "post": ("weight", "residual")}


def make(shape, form, dtype, wdtype, seed=0):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    D = shape[-1]
    d = dict(x=(rn(*shape) * 2).to(dtype), z=(2 * rn(*shape)).to(dtype), residual=rn(*shape).to(dtype), weight=(1 + 0.2 * rn(D)).to(wdtype),
             next_weight=(1 + 0.2 * rn(D)).to(wdtype), ds=rn(*shape).to(dtype), dy=rn(*shape).to(dtype))
    return {n: x if n in ("x", "ds") + FORMS[form] or (n == "dy" and "next_weight" in FORMS[form]) else None for n, x in d.items()}


def one_round(dtype):
    return T32 + (half(dtype) if dtype != F32 else 0)


def compare(d, act, alpha, eps, dtype, wdtype, g):
    names = ("x", "weight", "z", "residual", "next_weight")
    leaf = {n: d[n].double().requires_grad_() for n in names if d[n] is not None}
    s, y = norms(leaf["x"], leaf.get("weight"), leaf.get("z"), act, leaf.get("residual"), alpha, leaf.get("next_weight"), eps)
    kw = dict(weight=g["weight"], z=g["z"], act=act, residual=g["residual"], alpha=alpha, next_weight=g["next_weight"], eps=eps)
    gs, gy = norm_gate_fwd(g["x"], **kw)
    torch.cuda.synchronize()
    check("s", gs, s, one_round(dtype))
    assert (gy is None) == (y is None)
    if y is not None:
        check("y", gy, y, one_round(dtype))
    outs, cots = ([s], [d["ds"]]) if y is None else ([s, y], [d["ds"], d["dy"]])
    used = [n for n in names if n in leaf]
    # the gradient of the first norm's output, without its weight
    ds_all = torch.autograd.grad(outs, [s], [c.double() for c in cots], retain_graph=True)[0]
    gate = 1.0
    if "z" in leaf:
        zz = leaf["z"].detach()
        gate = torch.sigmoid(zz) if act == "sigmoid" else zz * torch.sigmoid(zz)
    ref_dn = alpha * ds_all * gate
    ref = dict(zip(used, torch.autograd.grad(outs, [leaf[n] for n in used], [c.double() for c in cots])))
    got = dict(zip(names, norm_gate_bwd(g["x"], g["ds"], g["dy"], **kw)))
    torch.cuda.synchronize()
    for n in names:
        assert (got[n] is None) == (n not in ref), n
        if n in ref:
            assert got[n].dtype == (wdtype if "weight" in n else dtype)
            more = 0.0
            if n == "x" and "weight" in leaf:
                x, up = leaf["x"].detach(), ref_dn
                more = T32 * float((up * leaf["weight"].detach() / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)).norm())
            check("d" + n, got[n], ref[n], one_round(got[n].dtype), more)


@pytest.mark.parametrize("dtype,wdtype", [(BF16, BF16), (BF16, F32), (F32, F32)], ids=str)
@pytest.mark.parametrize("form", FORMS)
def test_forms(form, dtype, wdtype):
    say(f"[case] norms {form} {dtype} {wdtype}")
    d = make((2, 3, 5, 64), form, dtype, wdtype, seed=1)
    g = {n: None if x is None else x.cuda() for n, x in d.items()}
    compare(d, "silu", 0.5, 1e-6, dtype, wdtype, g)
    compare(d, "sigmoid", -1.5, 1e-2, dtype, wdtype, g)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,D", [(1, 1), (3, 7), (700, 33), (17, 128), (5, 129), (33, 512), (9, 513), (6, 1024), (5, 1111), (4, 2048), (3, 4096),
                                    (7, 4100), (2, 8192), (3, 8193), (2, 16384), (1500, 256)])
def test_row_sizes(rows, D, dtype):
    say(f"[case] norms of {rows} rows of {D} {dtype}")
    d = make((rows, D), "block", dtype, F32, seed=2)
    g = {n: None if x is None else x.cuda() for n, x in d.items()}
    compare(d, "silu", 1.0, 1e-6, dtype, F32, g)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strided_rows(dtype):
    """Heads inside tokens, a slice that starts off 16 bytes, a broadcast gate."""
    say(f"[case] norms of strided rows {dtype}")
    d = make((2, 4, 6, 32), "block", dtype, F32, seed=3)
    g = {n: None if x is None else x.cuda() for n, x in d.items()}
    wide = torch.zeros(2, 6, 4, 35, dtype=dtype, device="cuda")
    wide[..., 1:33] = g["x"].transpose(1, 2)
    g["x"] = wide[..., 1:33].transpose(1, 2)
    g["residual"] = g["residual"].transpose(1, 2).contiguous().transpose(1, 2)
    d["z"] = d["z"][:, :1].expand(2, 4, 6, 32)
    g["z"] = d["z"][:, :1].cuda().expand(2, 4, 6, 32)
    compare(d, "sigmoid", 1.0, 1e-6, dtype, F32, g)


def test_rows_of_zeros_and_no_rows():
    say("[case] norms of zeros and of nothing")
    w = torch.ones(64, device="cuda")
    x = torch.zeros(3, 64, device="cuda")
    s, y = norm_gate_fwd(x, w, next_weight=w)
    dx, dw, _, _, dw2 = norm_gate_bwd(x, torch.ones_like(x), torch.ones_like(x), w, next_weight=w)
    assert (s == 0).all() and (y == 0).all() and torch.isfinite(dx).all() and (dw == 0).all() and (dw2 == 0).all()
    e = torch.empty(0, 64, device="cuda")
    s, _ = norm_gate_fwd(e, w)
    dx, dw = norm_gate_bwd(e, e, weight=w)[:2]
    torch.cuda.synchronize()
    assert s.shape == (0, 64) and dx.shape == (0, 64) and (dw == 0).all()


def test_a_row_does_not_reach_another():
    say("[case] norms, NaN in one row")
    d = make((40, 96), "block", BF16, F32, seed=4)
    g = {n: None if x is None else x.cuda() for n, x in d.items()}
    kw = {n: g[n] for n in ("weight", "z", "residual", "next_weight")}
    a = norm_gate_fwd(g["x"], **kw)
    g["x"][7] = float("nan")
    b = norm_gate_fwd(g["x"], **kw)
    rest = [i for i in range(40) if i != 7]
    assert all(torch.equal(p[rest], q[rest]) for p, q in zip(a, b)) and torch.isnan(b[0][7]).all()


def test_streams_and_graph_replays():
    say("[case] norms, side stream and graph")
    d = make((300, 4, 128), "block", BF16, F32, seed=5)
    g = {n: None if x is None else x.cuda() for n, x in d.items()}
    kw = {n: g[n] for n in ("weight", "z", "residual", "next_weight")}
    work = lambda **k: norm_gate_fwd(g["x"], **kw, **k) + norm_gate_bwd(g["x"], g["ds"], g["dy"], **kw, **k)  # noqa: E731
    ref = [x.clone() for x in work()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = work(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(ref, got))
    with torch.cuda.stream(side):
        work()
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
        assert all(torch.equal(x, y) for x, y in zip(work(), ref))
