"""The log-decay's gradient of heads that forget in one part of a sequence and remember in another, on the GPU against the
64-bit recurrence: every part is compared by itself, so that what is carried along the sequence may not bring the rounding of
a part whose values are large into one whose values are small.

Tolerances: dw of a token is a difference of sums over at most 16 chunks = 1024 tokens, sqrt(2 * 1024) = 45 times a product's
error (3 * 2^-17 where values are carried in two planes, 128 half steps in fp32), and in bf16 its own rounding, which is
taken from the reference itself."""
import math

import pytest

from gdr_testutil import check, gate_args, gpu
from kda_testutil import say
from lad_testutil import F32 as F32_TOL
from lad_testutil import SPLIT, make, reference

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from chunked_gated_delta_amd import lad_chunk_bwd  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
ROWS = ("q", "k", "v", "w", "dO")
FORGET, KEEP = -2.0, -1.0 / 2048

# (log-decay, share of the tokens) of the parts
PARTS = {
    "late": [(FORGET, 0.5), (KEEP, 0.5)],
    "early": [(KEEP, 0.5), (FORGET, 0.5)],
    "hill": [(FORGET, 0.3), (KEEP, 0.4), (FORGET, 0.3)],
    "valley": [(KEEP, 0.4), (FORGET, 0.2), (KEEP, 0.4)],
    "documents": [(KEEP, 0.4), (-math.inf, 0.0), (FORGET, 0.1), (-0.2, 0.1), (-math.inf, 0.0), (KEEP, 0.4)],
}


def decays(T, parts):
    """w of T tokens, and the parts' bounds; a part of no share is one token, counted with the next part."""
    w, bounds, at = torch.empty(T), [], 0
    for i, (g, share) in enumerate(parts):
        if share == 0.0:
            w[at] = g
            continue
        lo = bounds[-1][1] if bounds else 0
        hi = T if i + 1 == len(parts) else lo + int(share * T)
        keep = w[lo].item() if parts[i - 1][1] == 0.0 and i else None
        w[lo:hi] = g
        if keep is not None:
            w[lo] = keep
        bounds.append((lo, hi))
        at = hi
    return w, bounds


def inputs(B, T, H, dtype, kind, states):
    d = make(B, T, H, H, 64, 64, dtype, "log", seed=51, states=states)
    w, bounds = decays(T, PARTS[kind])
    d["w"] = w.to(dtype).expand(B, H, T).contiguous()
    return d, bounds


def compare(dw, ref, bounds, dtype):
    for lo, hi in bounds:
        r = ref[..., lo:hi]
        if dtype == F32:
            t = 45 * F32_TOL
        else:
            t = float((r.to(BF16).double() - r).norm()) / float(r.norm()) + 45 * SPLIT
        check(f"dw of tokens {lo} to {hi}", dw[..., lo:hi], r, t)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", PARTS)
@pytest.mark.parametrize("B,states", [(12, False), (12, True), (3, False)])
def test_parts_that_forget_and_remember(B, states, kind, dtype):
    """12 rows of 16 heads fill the machine with few segments a row, 3 with several."""
    say(f"[case] lad dw {B} rows {kind} states {states} {dtype}")
    T, H, of = 1500, 16, 2
    d, bounds = inputs(B, T, H, dtype, kind, B * states)
    t = gpu(d)
    got = lad_chunk_bwd(*(t[n] for n in ROWS), t["S0"], t["dS_final"], want_dS0=False, **gate_args("log"))
    torch.cuda.synchronize()
    one = {n: None if x is None else x[:1, :of] for n, x in d.items()}
    one["w"] = one["w"].clamp(min=-1e4)     # the same decays, with a finite derivative
    _, _, ref = reference(one, gate="log", grads=True)
    compare(got[3][:1, :of], ref["dw"], bounds, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", ["late", "early", "documents"])
def test_packed_sequences_that_forget_and_remember(kind, dtype):
    """Packed sequences of many heads, with entering states whose gradient is wanted."""
    say(f"[case] lad packed dw {kind} {dtype}")
    lens, H, of = [1100, 0, 400], 130, 1
    T = sum(lens)
    d, _ = inputs(1, T, H, dtype, kind, 3)
    w, bounds = decays(1100, PARTS[kind])
    d["w"][:, :, :1100] = w.to(dtype)
    t = gpu(d)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    got = lad_chunk_bwd(*(t[n] for n in ROWS), t["S0"], t["dS_final"], cu_seqlens=cu, **gate_args("log"))
    torch.cuda.synchronize()
    one = {n: x[:, :of] for n, x in d.items()}
    one["w"] = one["w"].clamp(min=-1e4)
    _, _, ref = reference(one, lens, gate="log", grads=True)
    compare(got[3][:, :of], ref["dw"], bounds + [(1100, T)], dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [130, 1100])
@pytest.mark.parametrize("empty", [("q", "k"), ("q",), ("k",)])
def test_tokens_that_neither_read_nor_write(empty, T, dtype):
    """Masked tokens (q or k zero, or both) between two states: dw is <S, R> alone, all of it behind a chunk that forgets nearly
    everything (e^-45)."""
    say(f"[case] lad dw of masked tokens {empty} {T} {dtype}")
    d = make(2, T, 2, 2, 64, 64, dtype, "log", seed=52, states=2)
    for n in empty:
        d[n].zero_()
    d["w"].fill_(-1.0 / 2048)
    d["w"][:, :, :64] = -0.7
    t = gpu(d)
    got = lad_chunk_bwd(*(t[n] for n in ROWS), t["S0"], t["dS_final"], **gate_args("log"))
    torch.cuda.synchronize()
    _, _, ref = reference(d, gate="log", grads=True)
    compare(got[3], ref["dw"], [(0, 64), (64, T)], dtype)
