"""The norms take any stride of their rows: they address each row in 64 bits, so the rule's limit on a token's stride
(64 tokens of a chunk within 32-bit offsets) is not theirs.  On the host by what the next check answers; on the
GPU with heads of a long [B,H,T,D] tensor taken token by token."""
import ctypes

import pytest
import torch

from chunked_gated_delta_amd import norm_gate_bwd, norm_gate_fwd
from gdr_testutil import check, half
from kda_testutil import say
from test_gdr_abi import P, dense, lib, nbwd, nfwd, norm_desc

FAR = 1 << 30                     # elements from one token to the next
TOO_FAR = dense(1, 1, 1, 1 << 46)   # past the 2^46 bytes that any tensor may reach: refused as a shape, -2


@pytest.mark.parametrize("name", ["x", "z", "residual"])
@pytest.mark.parametrize("dtype", [0, 1])
def test_far_rows_of_inputs_are_taken(name, dtype):
    """The call goes on to refuse the output that is out of reach."""
    far = dense(1, 1, 1, FAR)
    assert nfwd(norm_desc(T=2, dtype=dtype, **{name: far}), ss=TOO_FAR) == -2
    assert nbwd(norm_desc(T=2, dtype=dtype, **{name: far}), sx=TOO_FAR) == -2
    assert nfwd(norm_desc(T=2, dtype=dtype, **{name: TOO_FAR})) == -2


def test_far_rows_of_outputs_are_taken():
    d, far = norm_desc(T=2), dense(1, 1, 1, FAR)
    assert lib.kda_norm_fwd(P[0], P[1], P[2], P[3], P[4], ctypes.byref(d), P[5], ctypes.byref(far), P[6], ctypes.byref(TOO_FAR), None) == -2
    assert nbwd(d, sx=far, ws=None) == -4                 # the workspace is asked for after the strides


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")
@pytest.mark.parametrize("dtype,T", [(torch.bfloat16, 131073), (torch.float32, 65537)], ids=str)
def test_heads_of_a_long_tensor(dtype, T):
    """16 heads of T tokens, 32 MiB and a row from head to head, as [B,T,H,D]: every row equals that of the same
    tensor as it lies, and the weight's gradient (sums of 2^20 and 2^21 rows of random signs, at most 128 one behind
    another in a thread and 3 shorter sums behind those: 64 half steps of fp32) the one in 64 bits."""
    say(f"[case] norms of {T} x 16 rows across a long tensor, {dtype}")
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, z, ds = (torch.randn(1, 16, T, 128, generator=gen, device="cuda").to(dtype) for _ in range(3))
    w = torch.linspace(0.5, 1.5, 128, device="cuda")
    t = [a.transpose(1, 2) for a in (x, z, ds)]
    assert t[0].stride(2) * x.element_size() > 1 << 25
    s, _ = norm_gate_fwd(t[0], w, t[1])
    dx, dw, dz, _, _ = norm_gate_bwd(t[0], t[2], weight=w, z=t[1])
    s0, _ = norm_gate_fwd(x, w, z)
    dx0, dw0, dz0, _, _ = norm_gate_bwd(x, ds, weight=w, z=z)
    torch.cuda.synchronize()
    for far, near in ((s, s0), (dx, dx0), (dz, dz0)):
        assert far.shape == t[0].shape and torch.equal(far.transpose(1, 2), near)
    n = torch.zeros(128, dtype=torch.float64, device="cuda")
    for h in range(16):
        a, b, g = (y[:, h].double() for y in (x, z, ds))
        n += (g * b * torch.sigmoid(b) * a / torch.sqrt((a * a).mean(-1, keepdim=True) + 1e-6)).sum((0, 1))
    check("dw", dw, n.cpu(), 64 * half(torch.float32))
    check("dw as it lies", dw0, n.cpu(), 64 * half(torch.float32))
