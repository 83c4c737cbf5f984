"""Linear attention with a decay for each head where a chunk of 64 tokens holds many resets (several short documents behind
one another, set apart by a log-decay of -infinity), on the GPU against the 64-bit recurrence.

Between two resets a result is a sum over a few tokens, so its error is that of single products: in fp32 X . Y of 64
values and the products with Z, sqrt(64) half steps of fp32 each, and the decay's power, its scale and the products of
the three, 6 half steps: 22, taken as 32 half steps.  A reset adds 14427 to the prefixes (in units of ln 2), whose
differences have to stay as exact as they are without it."""
import math

import pytest

from gdr_testutil import check, gate_args, gpu
from kda_testutil import say
from lad_testutil import make, reference, tol

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from chunked_gated_delta_amd import lad_chunk_bwd, lad_chunk_fwd  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
NAMES = ("q", "k", "v", "w")
GRADS = ("dq", "dk", "dv", "dw", "dS0")
FEW = 32 * 2.0 ** -24


def with_resets(T, every, value, dtype, states=1):
    """A reset in every `every`-th token, decays of 0.05 to 0.15 between them."""
    d = make(1, T, 1, 2, 64, 64, dtype, "log", seed=41, states=states)
    gen = torch.Generator().manual_seed(42)
    d["w"] = -(0.05 + 0.1 * torch.rand(1, 2, T, generator=gen)).to(dtype)
    d["w"][:, :, every - 1::every] = value
    return d


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("value", [-math.inf, -1e4])
@pytest.mark.parametrize("every", [2, 3, 8, 32])
@pytest.mark.parametrize("T", [64, 333])
def test_many_resets_in_a_chunk(T, every, value, dtype):
    say(f"[case] lad {T} tokens, a reset every {every} {value} {dtype}")
    d = with_resets(T, every, value, dtype)
    t = gpu(d)
    o, S = lad_chunk_fwd(*(t[n] for n in NAMES), t["S0"], **gate_args("log"))
    got = lad_chunk_bwd(*(t[n] for n in NAMES), t["dO"], t["S0"], t["dS_final"], **gate_args("log"))
    torch.cuda.synchronize()
    ro, rS = reference(d, gate="log")
    few = FEW if dtype == F32 else 0.0
    check("o", o, ro, few or tol("o", dtype))
    check("S_final", S, rS, tol("S", dtype))
    e = {n: x.clone() for n, x in d.items()}
    e["w"].clamp_(min=-1e4)     # the same decays, with a finite derivative
    _, _, ref = reference(e, gate="log", grads=True)
    for n, x in zip(GRADS, got):
        check(n, x, ref[n], few if few and n in ("dq", "dk", "dv") else tol(n, dtype))
