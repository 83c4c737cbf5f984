"""Workspace sizes of no tokens and the largest launches of the head-gated delta rule, on the host."""
import ctypes

import pytest

import chunked_gated_delta_amd as kda
from test_gdr_abi import INVALID, bwd, desc, fwd, lib


@pytest.mark.parametrize("kw", [dict(dk=40), dict(dv=0), dict(Hk=0), dict(Hk=3), dict(B=0), dict(dtype=2), dict(gate=3), dict(g_min=1.0), dict(scale=float("inf")),
                                dict(B=2, n_seq=2)], ids=str)
@pytest.mark.parametrize("T", [0, 100])
def test_an_invalid_descriptor_has_no_size(kw, T):
    """As the header says, and whether or not there are tokens."""
    for backward in (0, 1):
        assert lib.kda_gdr_workspace_bytes(ctypes.byref(desc(T=T, **kw)), backward) == INVALID


def test_no_tokens_need_no_workspace():
    assert lib.kda_gdr_workspace_bytes(ctypes.byref(desc(T=0)), 1) == 0
    assert kda.gdr_workspace_bytes(1, 1, 2, 0, 64, 32) == kda.gdr_workspace_bytes(1, 1, 2, 0, 64, 32, n_seq=3, backward=True) == 0
    with pytest.raises(kda.KdaError):
        kda.gdr_workspace_bytes(1, 1, 2, 0, 64, 40)


def test_the_largest_launches():
    """A grid holds fewer than 2^32 threads.  The chains' workgroups of 512 are rounded up to eight units of
    (sequence, value head), the gradients' are one a chunk and key head: what would pass the limit is refused by its
    shape (-2) before anything is launched, what would not goes on to be refused by its missing workspace (-4)."""
    one = dict(Hk=1, Hv=1, dk=32, dv=32, T=1)
    assert fwd(desc(B=(1 << 22) - 8, **one), ws_bytes=0) == -4
    for B in ((1 << 22) - 7, (1 << 22) - 1, 1 << 22):
        assert fwd(desc(B=B, **one), ws_bytes=0) == -2, B
    # 2^23 chunks of 64 tokens, in one row
    far = dict(Hk=1, Hv=1, dk=32, dv=32, B=1)
    assert bwd(desc(T=64 * ((1 << 23) - 1), **far), ws_bytes=0) == -4
    assert bwd(desc(T=64 << 23, **far), ws_bytes=0) == -2
    assert fwd(desc(T=64 << 23, **far), ws_bytes=0) == -4     # its kernels of one workgroup a chunk have 256 threads
    assert lib.kda_gdr_workspace_bytes(ctypes.byref(desc(T=64 << 23, **far)), 0) != INVALID
    assert lib.kda_gdr_workspace_bytes(ctypes.byref(desc(T=64 << 23, **far)), 1) == INVALID
