"""Workspace sizes of no tokens of the head-gated delta rule, on the host."""
import ctypes

import pytest

import chunked_gated_delta_amd as kda
from test_gdr_abi import INVALID, desc, lib


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
