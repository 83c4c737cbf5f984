"""The workspace of linear attention holds what its calls write: the sizes against the segments' places on the host, and
calls on a workspace of exactly the size asked for, with guards around it, on the GPU."""
import ctypes
import random

import pytest
import torch

from chunked_gated_delta_amd import _lib, lad_chunk_bwd, lad_chunk_fwd
from chunked_gated_delta_amd._lib import KdaLad, KdaStride
from lad_testutil import make

lib = _lib.load()
CHUNK = 64


def section(n):
    return -(-int(n) // 256) * 256


def asked(B, T, Hv, n_seq, backward, dtype=1):
    z = KdaStride(0, 0, 0)
    d = KdaLad(B, Hv, Hv, T, 32, 32, n_seq, dtype, 2, 0, 0.0, 1.0, z, z, z, z)
    return lib.kda_lad_workspace_bytes(ctypes.byref(d), int(backward))


def bytes_of(slots, B, T, Hv, n_seq, backward):
    """What `slots` segments a head need, section by section, for 32 x 32 states."""
    state = 32 * 32 * 4
    n = section(slots * Hv * state) + section(slots * Hv * 4)
    if backward:
        n += section(slots * Hv * state) + section(slots * Hv * 4)     # adjoints and their decays
        n += 2 * section((n_seq or B) * Hv * state)                    # behind the last token, in front of the first
        n += 2 * section(2 * 8 * B * Hv * T) + section(8 * slots * Hv)  # dots in double, two kinds each; sums of a w per head
    return n


def slots_of(size, B, T, Hv, n_seq, backward):
    lo, hi = 0, T + (n_seq or B) + 1
    while lo < hi:      # the most segments that the size holds
        mid = (lo + hi + 1) // 2
        if bytes_of(mid, B, T, Hv, n_seq, backward) <= size:
            lo = mid
        else:
            hi = mid - 1
    return lo


def cuts(rng, T, n):
    kind = rng.randrange(4)
    if kind == 0:      # anywhere
        at = sorted(rng.randrange(T + 1) for _ in range(n - 1))
    elif kind == 1:    # one long sequence behind or in front of empty ones
        at = [rng.choice([0, T])] * (n - 1)
    elif kind == 2:    # one token over whole chunks
        at = sorted(min(T, CHUNK * rng.randrange(T // CHUNK + 1) + 1) for _ in range(n - 1))
    else:              # on whole chunks
        at = sorted(CHUNK * rng.randrange(T // CHUNK + 1) for _ in range(n - 1))
    return [0] + at + [T]


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("Hv", [1, 16, 130])
@pytest.mark.parametrize("T,n_seq", [(200, 1), (200, 7), (1024, 3), (1025, 200), (4099, 9), (70001, 5), (1 << 20, 1000)])
def test_packed_segments_fit(T, n_seq, Hv, backward):
    """A sequence at `start` has its segments from place floor(start / L) + its number on: for every segment length L that the
    size may stand for, all places lie inside it and no two sequences share one."""
    size = asked(1, T, Hv, n_seq, backward)
    rng = random.Random(T + n_seq + Hv)
    if size == 0:       # a forward whose segments hold whole sequences keeps nothing
        assert not backward
        return
    slots = slots_of(size, 1, T, Hv, n_seq, backward)
    assert bytes_of(slots, 1, T, Hv, n_seq, backward) == size
    lengths = [L for L in range(CHUNK, max(T, 3 * CHUNK) + CHUNK, CHUNK) if T // L + n_seq == slots]
    assert lengths, (size, slots)
    for L in {lengths[0], lengths[len(lengths) // 2], lengths[-1]}:
        for _ in range(40):
            cu, last = cuts(rng, T, n_seq), -1
            for i, (a, b) in enumerate(zip(cu, cu[1:])):
                first = a // L + i
                assert first > last
                last = first + max(1, -(-(b - a) // L)) - 1
                assert last < slots


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("B,T,Hv", [(1, 192, 1), (1, 193, 1), (3, 5000, 16), (12, 1500, 16), (2, 65536, 4), (1, 1 << 24, 1)])
def test_rows_segments_fit(B, T, Hv, backward):
    """Rows of a batch have ceil(T / L) segments each."""
    size = asked(B, T, Hv, 0, backward)
    if size == 0:
        assert not backward
        return
    slots = slots_of(size, B, T, Hv, 0, backward)
    assert bytes_of(slots, B, T, Hv, 0, backward) == size and slots >= B
    assert any(-(-T // L) * B == slots for L in range(CHUNK, T + 3 * CHUNK, CHUNK))


CALLS = [  # B, T, Hk, Hv, dk, dv, sequences
    (1, 700, 2, 4, 64, 32, [0, 300, 1, 399]),
    (1, 1500, 1, 1, 32, 64, [1, 1498, 1]),
    (1, 193, 1, 2, 32, 32, None),
    (3, 1100, 2, 2, 128, 128, None),
    (1, 130, 1, 4, 64, 64, [129, 0, 0, 1]),
]


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")
@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", CALLS, ids=str)
def test_calls_stay_inside(case, dtype, per_head):
    B, T, Hk, Hv, dk, dv, lens = case
    print(f"[case] lad workspace {case} {dtype} {per_head}", flush=True)
    n = len(lens) if lens else B
    d = {k: None if x is None else x.cuda() for k, x in make(B, T, Hk, Hv, dk, dv, dtype, "log", per_head, seed=61, states=n).items()}
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda() if lens else None
    args = [d[k] for k in ("q", "k", "v", "w")]
    for backward in (False, True):
        need = lib.kda_lad_workspace_bytes(ctypes.byref(KdaLad(B, Hk, Hv, T, dk, dv, len(lens) if lens else 0, int(dtype == torch.bfloat16), 2,
                                                                int(per_head), 0.0, 1.0, *[KdaStride(0, 0, 0)] * 4)), int(backward))
        guard = 1 << 20
        whole = torch.full((2 * guard + need,), 0xAB, dtype=torch.uint8, device="cuda")
        ws = whole[guard:guard + need] if need else None
        call = (lambda **k: lad_chunk_bwd(*args, d["dO"], d["S0"], d["dS_final"], log_decay=True, cu_seqlens=cu, **k)) if backward else \
            (lambda **k: lad_chunk_fwd(*args, d["S0"], log_decay=True, cu_seqlens=cu, **k))
        got, want = call(workspace=ws), call()
        torch.cuda.synchronize()
        assert (whole[:guard] == 0xAB).all() and (whole[guard + need:] == 0xAB).all()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
