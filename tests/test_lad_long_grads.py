"""Gradients of linear attention over long sequences, and decay gradients in fp32 at the accuracy that they have, on the GPU
against the 64-bit recurrence and its adjoint.

Tolerances of long sequences are test_lad.py's: a head that forgets within some hundred tokens sums no more than in a
short sequence.  A decay's gradient in fp32 is a sum over pairs of tokens taken from dots q.dq and k.dk, each of values that are
fp32 sums of up to 128 + 64 products with errors of their own sign, sqrt(192) = 14 half steps, over three planes where the inputs
are bf16 (2^-25, below that); d and e together 28: 32 half steps.  Two planes in place of three are off by 2^-17 and more,
four times that."""
import pytest

from gdr_testutil import check, gate_args, gpu, log_decay
from kda_testutil import say
from lad_testutil import make, reference, tol

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from chunked_gated_delta_amd import lad_chunk_bwd  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
ROWS = ("q", "k", "v", "w", "dO")
GRADS = ("dq", "dk", "dv", "dw", "dS0")
PAIRS = 32 * 2.0 ** -24
# A token's gradient is the sum of d - e over the tokens behind it in its chunk, 32 in the mean, up to 64, where the pairs of
# those tokens cancel and their errors do not: sqrt(2 * 32) = 8 times a dot's 14 half steps are 112, taken as 128.  (A head's
# is a sum over all tokens, in which each pair counts as often as there are tokens between its two: those far apart, of which
# there are many, carry it.)
TOKENS = 128 * 2.0 ** -24


def adjoint(d, gate):
    """Gradients by the recurrence and its adjoint, one batch row, no shared heads: S <- a S + k v^T, R <- a R + q dO^T backwards."""
    q, k, v, dO = (d[n][0].double().transpose(0, 1) for n in ("q", "k", "v", "dO"))      # [T, H, D]
    w = d["w"].double().requires_grad_()
    g = log_decay(w, gate)
    a = torch.exp(g.detach())[0].transpose(0, 1)
    T, H = q.shape[:2]
    S, old = d["S0"][0].double(), []
    dq, dk, dv, dg = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty(T, H, dtype=torch.float64)
    for t in range(T):
        old.append(a[t, :, None, None] * S)
        S = old[-1] + k[t, :, :, None] * v[t, :, None]
        dq[t] = (S * dO[t, :, None]).sum(-1)
    R = d["dS_final"][0].double()
    for t in reversed(range(T)):
        R = R + q[t, :, :, None] * dO[t, :, None]
        dk[t], dv[t] = (R * v[t, :, None]).sum(-1), (R * k[t, :, :, None]).sum(-2)
        dg[t] = (R * old.pop()).sum((-1, -2))
        R = a[t, :, None, None] * R
    dw, = torch.autograd.grad(g, w, dg.transpose(0, 1)[None])
    return {"dq": dq.transpose(0, 1)[None], "dk": dk.transpose(0, 1)[None], "dv": dv.transpose(0, 1)[None], "dw": dw, "dS0": R[None]}


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,H,D", [(8200, 2, 64), (30000, 1, 32)])
def test_long_sequences(T, H, D, dtype):
    say(f"[case] lad gradients of {T} tokens {dtype}")
    d = make(1, T, H, H, D, D, dtype, "log", seed=71, states=1)
    d["w"] = (0.02 * d["w"].float()).to(dtype)
    t = gpu(d)
    got = lad_chunk_bwd(*(t[n] for n in ROWS), t["S0"], t["dS_final"], **gate_args("log"))
    torch.cuda.synchronize()
    ref = adjoint(d, "log")
    for n, x in zip(GRADS, got):
        check(n, x, ref[n], tol(n, dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,T,dk,dv,states", [(1, 130, 128, 128, False), (2, 700, 64, 128, True), (2, 700, 128, 128, False)])
def test_decay_gradients_of_heads(B, T, dk, dv, states, dtype):
    """One decay a head: its gradient is in fp32, also of bf16 inputs."""
    say(f"[case] lad dw of heads {B} {T} {dk} {dv} {states} {dtype}")
    d = make(B, T, 4, 8, dk, dv, dtype, "log", per_head=True, seed=72, states=B * states)
    t = gpu(d)
    got = lad_chunk_bwd(*(t[n] for n in ROWS), t["S0"], t["dS_final"], **gate_args("log"))
    torch.cuda.synchronize()
    check("dw", got[3], reference(d, gate="log", grads=True)[2]["dw"], PAIRS)


@pytest.mark.parametrize("gate", ["bounded", "softplus"])
@pytest.mark.parametrize("B,T", [(1, 150), (3, 700)])
def test_decay_gradients_of_tokens_in_fp32(B, T, gate):
    say(f"[case] lad dw of tokens {B} {T} {gate}")
    d = make(B, T, 2, 4, 64, 128, F32, gate, seed=73, states=B)
    t = gpu(d)
    got = lad_chunk_bwd(*(t[n] for n in ROWS), t["S0"], t["dS_final"], **gate_args(gate))
    torch.cuda.synchronize()
    check("dw", got[3], reference(d, gate=gate, grads=True)[2]["dw"], TOKENS)
