"""Calls of linear attention and of the norms with rotation that the documentation allows and that are out of the
ordinary: tokens in front of the first sequence, one tensor for several inputs, broadcast inputs and gradients, on the
GPU against the 64-bit forms.  Tolerances as in test_lad.py and test_qk_norm.py."""
import pytest

from gdr_testutil import check, gate_args, gpu, half
from kda_testutil import say
from lad_testutil import make, reference, rotate, tol

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from chunked_gated_delta_amd import lad_chunk_bwd, lad_chunk_fwd, lad_decode, qk_norm_rope_bwd, qk_norm_rope_fwd  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
NAMES = ("q", "k", "v", "w")
GRADS = ("dq", "dk", "dv", "dw", "dS0")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("per_head", [False, True])
def test_tokens_in_front_of_the_first_sequence(per_head, dtype):
    """Offsets that start behind 0 and end before T: the rest of an output is left as it was, and NaN there reach nothing."""
    say(f"[case] lad offsets from 5 {per_head} {dtype}")
    lo, lens, T = 5, [65, 0, 230], 320
    hi = lo + sum(lens)
    d = make(1, T, 1, 2, 64, 32, dtype, per_head=per_head, seed=31, states=3)
    rows = [n for n in ("q", "k", "v", "w", "dO") if d[n].dim() > 1]
    inside = dict(d, **{n: d[n][:, :, lo:hi] for n in rows})
    for n in rows:
        d[n] = d[n].clone()
        d[n][:, :, :lo] = d[n][:, :, hi:] = float("nan")
    t = gpu(d)
    cu = torch.tensor([lo, lo + 65, lo + 65, hi], dtype=torch.int32, device="cuda")
    out = torch.full((1, 2, T, 32), 3.0, dtype=dtype, device="cuda")
    o, S = lad_chunk_fwd(*(t[n] for n in NAMES), t["S0"], cu_seqlens=cu, out=out)
    got = lad_chunk_bwd(*(t[n] for n in NAMES), t["dO"], t["S0"], t["dS_final"], cu_seqlens=cu)
    torch.cuda.synchronize()
    assert (o[:, :, :lo] == 3).all() and (o[:, :, hi:] == 3).all()
    ro, rS, ref = reference(inside, lens, grads=True)
    check("o", o[:, :, lo:hi], ro, tol("o", dtype))
    check("S", S, rS, tol("S", dtype))
    for n, g in zip(GRADS, got):
        check(n, g[:, :, lo:hi] if n in ("dq", "dk", "dv") or (n == "dw" and not per_head) else g, ref[n], tol(n, dtype, per_head))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [100, 400])
def test_one_tensor_for_several_inputs(T, dtype):
    """q and k the same tensor, v one head for all, dO one row of the batch for all."""
    say(f"[case] lad with q = k and broadcasts {T} {dtype}")
    B, H, D = 2, 3, 64
    d = make(B, T, H, H, D, D, dtype, gate="log", seed=32)
    d["k"] = d["q"]
    d["v"] = d["v"][:, :1].expand(B, H, T, D)
    d["dO"] = d["dO"][:1].expand(B, H, T, D)
    t = gpu({n: d[n] for n in ("q", "w")})
    t["k"] = t["q"]
    t["v"] = d["v"][:, :1].cuda().expand(B, H, T, D)
    t["dO"] = d["dO"][:1].cuda().expand(B, H, T, D)
    o, S = lad_chunk_fwd(*(t[n] for n in NAMES), **gate_args("log"))
    got = lad_chunk_bwd(*(t[n] for n in NAMES), t["dO"], **gate_args("log"))
    torch.cuda.synchronize()
    full = dict(d, k=d["k"].clone(), v=d["v"].clone(), dO=d["dO"].clone())
    ro, rS, ref = reference(full, gate="log", grads=True)
    check("o", o, ro, tol("o", dtype))
    check("S", S, rS, tol("S", dtype))
    for n, g in zip(GRADS[:4], got):
        check(n, g, ref[n], tol(n, dtype))


def test_many_heads():
    """More heads than workgroups that run at once, with several segments each."""
    say("[case] lad with 600 heads")
    d = make(1, 260, 600, 600, 32, 32, BF16, seed=33)
    t = gpu(d)
    o, S = lad_chunk_fwd(*(t[n] for n in NAMES))
    got = lad_chunk_bwd(*(t[n] for n in NAMES), t["dO"])
    torch.cuda.synchronize()
    ro, rS, ref = reference(d, grads=True)
    check("o", o, ro, tol("o", BF16))
    check("S", S, rS, tol("S", BF16))
    for n, g in zip(GRADS[:4], got):
        check(n, g, ref[n], tol(n, BF16))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_step_of_broadcast_rows(dtype):
    """The same token for every row of a pool, and a state of which no row is the first."""
    say(f"[case] lad step of broadcast rows {dtype}")
    B, T, H, D, dv = 5, 3, 2, 64, 128
    d = make(1, T, H, H, D, dv, dtype, seed=34, states=4)
    t = gpu(d)
    wide = {n: t[n].expand(B, *t[n].shape[1:]) for n in NAMES}
    slots = torch.tensor([2, -1, 0, 2, 4], dtype=torch.int32, device="cuda")   # 4: behind the pool
    S = t["S0"].clone()
    o = lad_decode(*(wide[n] for n in NAMES), S, slots)
    torch.cuda.synchronize()
    assert torch.equal(S[1], t["S0"][1]) and torch.equal(S[3], t["S0"][3])
    assert (o[1] == 0).all() and (o[4] == 0).all()
    one, two = dict(d, S0=d["S0"][:1]), dict(d, S0=d["S0"][2:3])
    twice = dict(two, **{n: torch.cat([d[n], d[n]], 2) for n in NAMES})
    ro, rS = reference(one)
    check("o of row 2", o[2:3], ro, tol("o", dtype))
    check("S of slot 0", S[:1], rS, tol("S", dtype))
    ro, rS = reference(twice)
    check("o of rows 0, 3", torch.cat([o[:1], o[3:4]], 2), ro, tol("o", dtype))
    check("S of slot 2", S[2:3], rS, tol("S", dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("near", [False, True])
def test_rotation_of_one_tensor_twice(near, dtype):
    """q and k the same tensor at different scales, one head for all of them, and one gradient for all heads."""
    say(f"[case] qk norm of broadcast rows {near} {dtype}")
    B, T, H, D, R = 2, 37, 3, 80, 32
    gen = torch.Generator().manual_seed(35)
    x, dy = torch.randn(B, 1, T, D, generator=gen).to(dtype), torch.randn(1, 1, T, D, generator=gen).to(dtype)
    w, positions = 1 + 0.1 * torch.randn(D, generator=gen), torch.arange(T)[None] - 20
    inv_freq = (1e4 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)).float()
    q, g = x.cuda().expand(B, H, T, D), dy.cuda().expand(B, H, T, D)
    pos = positions.cuda().expand(B, T)
    kw = dict(interleaved=near, q_scale=0.5, k_scale=2.0)
    out = qk_norm_rope_fwd(q, q, w.cuda(), w.cuda(), pos, inv_freq.cuda(), **kw)
    got = qk_norm_rope_bwd(q, q, g, g, w.cuda(), w.cuda(), pos, inv_freq.cuda(), **kw)
    torch.cuda.synchronize()
    own = half(dtype) if dtype == BF16 else 0.0
    for y, dx, dw, scale in ((out[0], got[0], got[2], 0.5), (out[1], got[1], got[3], 2.0)):
        xr, wr = x.double().expand(B, H, T, D).clone().requires_grad_(), w.double().requires_grad_()
        ref = rotate(xr, wr, positions, inv_freq, interleaved=near, scale=scale)
        rx, rw = torch.autograd.grad(ref, (xr, wr), dy.double().expand(B, H, T, D))
        check("y", y, ref, own + 32 * 2.0 ** -24)
        check("dx", dx, rx, own + 64 * 2.0 ** -24)
        check("dw", dw, rw, 128 * 2.0 ** -24)
