"""Final states and the entering states' gradients of the head-gated delta rule for bf16 inputs: they are fp32
results of fp32 accuracy, since what the chains compute (S, E, T', U; dS, X, P, T^T, gam dO, gam dE) enters the matrix
cores in three bf16 planes.

Tolerance, in half steps of fp32, 2-norm relative: a sum of n products of random signs, rounded after each, is off by
sqrt(n / 6) of them (roundings uniform in half a step, 1 / sqrt(3) of it each, of partial sums that grow as
sqrt(i)): 4.6 for 128 products, 3.3 for 64.  S_final: K S (128), the solve for T', T' E and K^T U (64 each), added up 14.5;
four operands of three planes, each off by 2^-25, half a half step: 2.  17 in all, 1.0e-6.  dS0: K dS (128),
the solve, P^T dO, T^T X, Q^T gam dO and K^T gam dE (64 each), 21; six operands, 3.  24 in all, 1.4e-6.

Two planes (off by 2^-17) of the operands that weigh most, U and gam dO, are off by 2e-6 and more, and a test on the CPU
shows that of a 64-bit chunk form; two planes of S, T', dS or T^T alone stay below these bounds."""
import pytest
import torch

from gdr_testutil import check, gate_args, gpu, half, log_decay, make, reference
from kda_testutil import say

TOL_S, TOL_DS0 = 17 * half(torch.float32), 24 * half(torch.float32)
CASES = [  # B, T, Hk, Hv, dk, dv, gate
    (1, 130, 2, 2, 128, 128, "bounded"), (2, 300, 1, 2, 64, 128, "softplus"), (1, 200, 2, 2, 128, 64, "log"), (3, 64, 1, 2, 32, 32, "bounded"),
    (1, 200, 1, 2, 128, 128, "slow")]


def inputs(case):
    B, T, Hk, Hv, dk, dv, gate = case
    d = make(B, T, Hk, Hv, dk, dv, torch.bfloat16, "log" if gate == "slow" else gate, seed=60, states=B)
    if gate == "slow":   # hardly any decay, keys that lean one way, small rates: old states weigh
        gen = torch.Generator().manual_seed(61)
        way = torch.randn(dk, generator=gen, dtype=torch.float64)
        for n in ("q", "k"):
            x = d[n].double() + way / way.norm()
            d[n] = (x / x.norm(dim=-1, keepdim=True)).to(torch.bfloat16)
        d["w"] = (-0.01 * torch.rand(d["w"].shape, generator=gen)).to(torch.bfloat16)
        d["beta"] = (0.05 + 0.3 * torch.rand(d["beta"].shape, generator=gen)).to(torch.bfloat16)
    return d, "log" if gate == "slow" else gate


def in_planes(x, n):
    """x as a sum of n bf16 values."""
    total = torch.zeros_like(x)
    for _ in range(n):
        h = (x - total).to(torch.bfloat16).double()
        total = total + h
    return total


def chunk_form(d, gate, coarse=()):
    """S_final and dS0 by chunks of 64 in 64 bits, each computed operand in three planes, those of `coarse` in two."""
    of = lambda name, x: in_planes(x, 2 if name in coarse else 3)  # noqa: E731
    tr = lambda x: x.transpose(-1, -2)  # noqa: E731
    grp = d["v"].shape[1] // d["q"].shape[1]
    q, k = (d[n].double().repeat_interleave(grp, 1) for n in ("q", "k"))
    v, beta, dO, g = d["v"].double(), d["beta"].double(), d["dO"].double(), log_decay(d["w"].double(), gate)
    S, chunks = d["S0"].double(), []
    for a in range(0, q.shape[2], 64):
        K, Q, V, b, do, G = (x[:, :, a:a + 64] for x in (k, q, v, beta, dO, g))
        b, G = b[..., None], G.cumsum(-1)
        D = torch.exp(G[..., :, None] - G[..., None, :]).tril()
        gam, eta, last = G.exp()[..., None], (G[..., -1:] - G).exp()[..., None], G[..., -1].exp()[..., None, None]
        A, eye = (K @ tr(K) * D).tril(-1), torch.eye(K.shape[2], dtype=torch.float64)
        U = b * (of("T", torch.linalg.inv(eye + A * tr(b))) @ of("E", V - gam * (K @ of("S", S))))
        S = last * S + tr(K) @ of("U", eta * U)
        chunks.append((K, Q, b, do, gam, eta, last, tr(torch.linalg.inv(eye + b * A)), tr(Q @ tr(K) * D)))
    dS = d["dS_final"].double()
    for K, Q, b, do, gam, eta, last, Tt, P in reversed(chunks):
        dU = of("Tt", Tt) @ of("X", of("P", P) @ do + eta * (K @ of("dS", dS)))
        dS = last * dS + tr(Q) @ of("dO", gam * do) + tr(K) @ of("dE", -gam * b * dU)
    return S, dS


def off(x, ref):
    return float((x - ref).norm() / ref.norm())


@pytest.mark.parametrize("case", CASES, ids=str)
def test_the_tolerance_tells_two_planes_from_three(case):
    d, gate = inputs(case)
    _, S, ref = reference(d, gate=gate, grads=True)
    S = S.detach()
    fine, coarse = chunk_form(d, gate), chunk_form(d, gate, ("S", "T", "E", "U", "P", "dS", "Tt", "X", "dO", "dE"))
    print(f"   three planes {off(fine[0], S):.1e} {off(fine[1], ref['dS0']):.1e}, two {off(coarse[0], S):.1e} {off(coarse[1], ref['dS0']):.1e}")
    assert off(fine[0], S) < TOL_S / 20 and off(fine[1], ref["dS0"]) < TOL_DS0 / 20
    assert off(coarse[0], S) > TOL_S and off(coarse[1], ref["dS0"]) > TOL_DS0
    if case[-1] != "slow":
        assert off(chunk_form(d, gate, ("U",))[0], S) > TOL_S and off(chunk_form(d, gate, ("dO",))[1], ref["dS0"]) > TOL_DS0


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")
@pytest.mark.parametrize("case", CASES, ids=str)
def test_states_of_bf16_inputs(case):
    from chunked_gated_delta_amd import gdr_chunk_bwd, gdr_chunk_fwd
    say(f"[case] gdr states {case}")
    d, gate = inputs(case)
    _, S, ref = reference(d, gate=gate, grads=True)
    t, names = gpu(d), ("q", "k", "v", "w", "beta")
    got = gdr_chunk_fwd(*(t[n] for n in names), t["S0"], **gate_args(gate))[1]
    dS0 = gdr_chunk_bwd(*(t[n] for n in names), t["dO"], t["S0"], t["dS_final"], **gate_args(gate))[5]
    torch.cuda.synchronize()
    check("S_final", got, S, TOL_S)
    check("dS0", dS0, ref["dS0"], TOL_DS0)
