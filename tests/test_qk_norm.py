"""Norms of queries and keys with the rotation by position, on the GPU, against their 64-bit form.

Tolerances: a row's square sum is 16 products a lane and up to 6 sums over lanes, the norm, the weight, the scale and the
rotation 8 operations more, the angle's sine and cosine 2 half steps of 1: 32 half steps of fp32, doubled for the
gradient, which takes a second such sum, and the results' own rounding.  Weights' gradients are sums over rows, in
registers, lanes, wavefronts and workgroups one after another: another 64 half steps."""
import pytest

from gdr_testutil import check, half
from kda_testutil import say
from lad_testutil import rotate

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from chunked_gated_delta_amd import KdaError, gdr_chunk_fwd, lad_chunk_bwd, lad_chunk_fwd, norm_gate_fwd, qk_norm_rope_bwd, qk_norm_rope_fwd  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
FWD, BWD, SUMS = 32 * 2.0 ** -24, 64 * 2.0 ** -24, 128 * 2.0 ** -24


def own(dtype):
    return half(dtype) if dtype == BF16 else 0.0


CASES = [  # B, T, Hq, Hk, D, R, norm, weight type ("": none), interleaved, positions, layout
    (1, 1, 1, 1, 2, 2, True, F32, False, "row", "head"),
    (2, 7, 3, 1, 64, 64, True, BF16, False, "each", "token"),
    (1, 130, 4, 2, 128, 128, True, F32, False, "wide", "fused"),
    (3, 33, 2, 2, 128, 64, True, BF16, True, "each", "token"),
    (1, 65, 5, 1, 80, 36, True, F32, True, "row", "head"),
    (1, 50, 2, 1, 80, 36, True, F32, False, "row", "odd"),
    (2, 19, 2, 1, 96, 96, False, F32, False, "each", "token"),
    (1, 40, 2, 2, 256, 32, True, "", False, "far", "token"),
    (1, 9, 1, 1, 512, 512, True, F32, True, "row", "head"),
    (1, 5, 2, 1, 1024, 1024, True, BF16, False, "each", "fused"),
    (1, 6, 2, 1, 1000, 998, True, F32, False, "row", "odd"),
    (2, 21, 3, 3, 128, 0, True, F32, False, "", "token"),
    (2, 21, 3, 3, 32, 32, False, "", False, "each", "fused"),
    (1, 3000, 4, 4, 64, 64, True, F32, False, "row", "token"),
    (1, 77, 3, 0, 128, 128, True, F32, False, "row", "token"),
    (2, 40, 2, 1, 128, 52, True, BF16, False, "each", "odd"),
    (1, 33, 3, 1, 96, 24, True, F32, False, "row", "token"),
    (1, 33, 2, 1, 100, 36, True, F32, True, "row", "odd"),
    (1, 70, 1, 1, 128, 122, True, F32, False, "row", "head"),
    (1, 30, 1, 1, 48, 16, True, F32, False, "row", "fused"),
    (1, 30, 2, 1, 1024, 514, True, F32, False, "row", "token"),
    (1, 20, 1, 1, 384, 100, True, "", False, "row", "token"),
]


def make(case, dtype, seed=0):
    B, T, Hq, Hk, D, R, norm, wt, near, pos, layout = case
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731

    def rows(H):
        x = (rn(B, T, H, D) * torch.exp(0.5 * rn(B, T, H, 1))).to(dtype)
        if layout == "head":
            return x.transpose(1, 2).contiguous()
        if layout == "odd":      # rows at odd places
            buf = torch.zeros(B, T, H, D + 3, dtype=dtype)
            buf[..., 1:D + 1] = x
            return buf[..., 1:D + 1].transpose(1, 2)
        return x.transpose(1, 2)

    d = dict(q=rows(Hq), k=rows(Hk) if Hk else None, dq=rows(Hq), dk=rows(Hk) if Hk else None)
    if layout == "fused":
        x = torch.cat([d["q"].transpose(1, 2).flatten(2), d["k"].transpose(1, 2).flatten(2)], -1)
        d["q"], d["k"] = x[..., :Hq * D].unflatten(-1, (Hq, D)).transpose(1, 2), x[..., Hq * D:].unflatten(-1, (Hk, D)).transpose(1, 2)
    for n in ("q_weight", "k_weight"):
        d[n] = (1 + 0.1 * rn(D)).to(wt) if wt != "" and (n == "q_weight" or Hk) else None
    d["positions"] = {"": None, "row": torch.arange(T, dtype=torch.int32), "wide": torch.arange(T, dtype=torch.int64)[None] + 5_000_000_000,
                      "each": torch.randint(-50, 5000, (B, T), generator=gen, dtype=torch.int32),
                      "far": torch.randint(0, 1 << 24, (B, T), generator=gen, dtype=torch.int32)}[pos]
    d["inv_freq"] = (1e4 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)).float() if R else None
    return d


def cuda(x):
    """On the GPU, strides kept."""
    if x is None:
        return None
    if x.dim() < 4:
        return x.cuda()
    base = x._base if x._base is not None else x
    while base._base is not None:
        base = base._base
    return torch.as_strided(base.cuda(), x.shape, x.stride(), x.storage_offset())


def call(case):
    norm, near = case[6], case[8]
    return dict(norm=norm, interleaved=near, q_scale=0.125, k_scale=1.5)


def plain(d, case, n, x=None):
    return rotate(d[n].double() if x is None else x, d[n + "_weight"].double() if d[n + "_weight"] is not None else None, d["positions"],
                  d["inv_freq"], case[6], case[8], 0.125 if n == "q" else 1.5)


def takes(case):
    return case[6] or case[7] != "" or case[5] > 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(case, dtype):
    say(f"[case] qk norm forward {case} {dtype}")
    d = make(case, dtype, 1)
    t = {n: cuda(x) for n, x in d.items()}
    out = qk_norm_rope_fwd(t["q"], t["k"], t["q_weight"], t["k_weight"], t["positions"], t["inv_freq"], **call(case))
    torch.cuda.synchronize()
    for n, x in zip("qk", out):
        if d[n] is None:
            assert x is None
            continue
        assert x.dtype == dtype
        check(n, x, plain(d, case, n), own(dtype) + FWD)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(case, dtype):
    say(f"[case] qk norm backward {case} {dtype}")
    d = make(case, dtype, 2)
    t = {n: cuda(x) for n, x in d.items()}
    got = qk_norm_rope_bwd(t["q"], t["k"], t["dq"], t["dk"], t["q_weight"], t["k_weight"], t["positions"], t["inv_freq"], **call(case))
    torch.cuda.synchronize()
    for n, gx, gw in (("q", got[0], got[2]), ("k", got[1], got[3])):
        if d[n] is None:
            assert gx is None and gw is None
            continue
        x = d[n].double().requires_grad_()
        w = d[n + "_weight"].double().requires_grad_() if d[n + "_weight"] is not None else None
        y = rotate(x, w, d["positions"], d["inv_freq"], case[6], case[8], 0.125 if n == "q" else 1.5)
        ref = torch.autograd.grad(y, [x] + ([w] if w is not None else []), d["d" + n].double())
        # a row of one pair: what the norm leaves of the gradient is a difference of equal terms
        size = float(d["d" + n].double().norm()) if case[4] == 2 else 0.0
        check("d" + n, gx, ref[0], own(dtype) + BWD, more=BWD * size)
        assert (gw is None) == (w is None)
        if w is not None:
            assert gw.dtype == d[n + "_weight"].dtype
            check("d" + n + "_weight", gw, ref[1], own(gw.dtype) + SUMS)


def test_rows_without_anything():
    """A row of zeros stays zero and has finite gradients; no tokens give empty rows and zero weight gradients."""
    say("[case] qk norm of zeros and of nothing")
    q = torch.zeros(1, 2, 5, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    pos, freq = torch.arange(5, dtype=torch.int32, device="cuda"), torch.ones(32, device="cuda")
    y, _ = qk_norm_rope_fwd(q, None, w, None, pos, freq)
    assert (y == 0).all()
    g = qk_norm_rope_bwd(q, None, torch.ones_like(q), None, w, None, pos, freq)
    assert torch.isfinite(g[0]).all() and (g[2] == 0).all()
    e = torch.zeros(1, 2, 0, 64, device="cuda")
    y, k = qk_norm_rope_fwd(e, e, w, w, pos[:0], freq)
    assert y.shape == e.shape and k.shape == e.shape
    g = qk_norm_rope_bwd(e, e, e, e, w, w, pos[:0], freq)
    assert (g[2] == 0).all() and (g[3] == 0).all()


def test_a_row_with_a_nan_stays_alone():
    say("[case] qk norm with a NaN")
    q = torch.randn(1, 3, 40, 128, device="cuda")
    q[0, 1, 7, 5] = float("nan")
    q[0, 2, 8, 127] = float("inf")
    y, _ = qk_norm_rope_fwd(q, None, positions=torch.arange(40, dtype=torch.int32, device="cuda"), inv_freq=torch.ones(64, device="cuda"))
    bad = ~torch.isfinite(y).all(-1)
    assert bad.sum() == 2 and bad[0, 1, 7] and bad[0, 2, 8]


def test_gradients_against_differences():
    say("[case] qk norm differences")
    case = (1, 9, 2, 1, 32, 16, True, F32, False, "row", "head")
    d = make(case, F32, 3)
    t = {n: cuda(x) for n, x in d.items()}
    got = qk_norm_rope_bwd(t["q"], t["k"], t["dq"], t["dk"], t["q_weight"], t["k_weight"], t["positions"], t["inv_freq"], **call(case))
    grads = dict(zip(("q", "k", "q_weight", "k_weight"), got))

    def loss(e):
        out = qk_norm_rope_fwd(e["q"], e["k"], e["q_weight"], e["k_weight"], e["positions"], e["inv_freq"], **call(case))
        return sum(float((y.double() * e["d" + n].double()).sum()) for n, y in zip("qk", out))

    gen = torch.Generator().manual_seed(4)
    h = 2.0 ** -6
    for n, g in grads.items():
        u = torch.randn(d[n].shape, generator=gen)
        u = (u / u.norm()).cuda()
        by_diff = (loss(dict(t, **{n: t[n] + h * u})) - loss(dict(t, **{n: t[n] - h * u}))) / (2 * h)
        by_grad = float((g.double() * u.double()).sum())
        # the loss sums 900 products of size 1 off by 32 half steps each: 6e-5 at most, over 2 h; the third derivative by h^2
        assert abs(by_diff - by_grad) <= 2e-3 * float(g.double().norm()) + 3e-5 / h


def test_outputs_where_they_are_wanted():
    """Outputs into slices of buffers, whose rest stays; two outputs whose spans meet are refused, as documented."""
    say("[case] qk norm outputs")
    q, k = torch.randn(2, 4, 30, 64, device="cuda").to(BF16), torch.randn(2, 2, 30, 64, device="cuda").to(BF16)
    buf = torch.full((2, 30, 8, 64), 9.0, dtype=BF16, device="cuda")
    qo, ko = buf[:, :, :4].transpose(1, 2), buf[:, :, 4:6].transpose(1, 2)
    with pytest.raises(KdaError, match="code -4"):
        qk_norm_rope_fwd(q, k, q_out=qo, k_out=ko)
    other = torch.full((2, 30, 3, 64), 9.0, dtype=BF16, device="cuda")
    ko = other[:, :, 1:].transpose(1, 2)
    a, b = qk_norm_rope_fwd(q, k, q_out=qo, k_out=ko)
    c, e = qk_norm_rope_fwd(q, k)
    assert a is qo and b is ko and torch.equal(a, c) and torch.equal(b, e)
    assert (buf[:, :, 4:] == 9).all() and (other[:, :, 0] == 9).all()


def test_a_layer_of_them():
    """Norm and rotation, linear attention with a decay, the heads' gated norm, and the gradients back to the projection, as a
    layer runs them; and the delta rule on the same unit rows."""
    say("[case] norm and rotation, linear attention, gated norm")
    B, T, Hq, Hv, D = 1, 190, 2, 4, 64
    gen = torch.Generator().manual_seed(5)
    x = torch.randn(B, T, (2 * Hq + 2 * Hv) * D, generator=gen)
    w = torch.linspace(-0.5, -0.01, Hv)
    gain, qw, kw = (1 + 0.1 * torch.randn(D, generator=gen) for _ in range(3))
    pos, freq = torch.arange(T, dtype=torch.int32), (1e4 ** (-torch.arange(0, D, 2) / D)).float()
    dO = torch.randn(B, Hv, T, D, generator=gen)

    def split(x):
        cut = x.split([Hq * D, Hq * D, Hv * D, Hv * D], -1)
        return [c.unflatten(-1, (-1, D)).transpose(1, 2) for c in cut]

    q, k, v, z = split(x.cuda())
    args = (qw.cuda(), kw.cuda(), pos.cuda(), freq.cuda())
    qn, kn = qk_norm_rope_fwd(q, k, *args, k_scale=D ** -0.5)
    o, S = lad_chunk_fwd(qn, kn, v, w.cuda(), scale=D ** -0.5, log_decay=True)
    y, _ = norm_gate_fwd(o, gain.cuda(), z)
    dqn, dkn, dv, dw, _ = lad_chunk_bwd(qn, kn, v, w.cuda(), dO.cuda(), scale=D ** -0.5, log_decay=True)
    dq, dk, dqw, dkw = qk_norm_rope_bwd(q, k, dqn, dkn, *args, k_scale=D ** -0.5)

    from gdr_testutil import norms, rule as gdr_rule
    from lad_testutil import rule
    leaves = [t.double().requires_grad_() for t in (x, qw, kw, w)]
    q6, k6, v6, z6 = split(leaves[0])
    qn6 = rotate(q6, leaves[1], pos, freq)
    kn6 = rotate(k6, leaves[2], pos, freq, scale=D ** -0.5)
    o6, S6 = rule(qn6, kn6, v6, leaves[3], gate="log", scale=D ** -0.5)
    y6, _ = norms(o6, gain.double(), z6)
    F32_SUM = 128 * 2.0 ** -24
    check("y", y, y6, 2 * F32_SUM)
    check("S", S, S6, 2 * F32_SUM)
    (o6 * dO.double()).sum().backward()
    gq, gk, gv, _ = split(leaves[0].grad)
    for n, a, b in (("dq", dq, gq), ("dk", dk, gk), ("dv", dv, gv), ("dq_weight", dqw, leaves[1].grad), ("dk_weight", dkw, leaves[2].grad)):
        check(n, a, b, 3 * F32_SUM)
    check("dw", dw, leaves[3].grad, 32 * F32_SUM)
    beta = torch.full((B, Hv, T), 0.5)
    og, _ = gdr_chunk_fwd(qn, kn, v, w.cuda().view(1, Hv, 1).expand(B, Hv, T).contiguous(), beta.cuda(), log_decay=True)
    plain_kn = rotate(k6.detach(), kw.double(), pos, freq, scale=D ** -0.5)
    plain_qn = rotate(q6.detach(), qw.double(), pos, freq)
    ref, _ = gdr_rule(plain_qn, plain_kn, v6.detach(), w.double().view(1, Hv, 1).expand(B, Hv, T), beta.double(), gate="log")
    check("o of the delta rule", og, ref, 2 * F32_SUM)
