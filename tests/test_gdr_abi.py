"""Refusals of the head-gated delta rule and of the norms around a block, on the host: every invalid call
returns its code before any HIP call (so these run without a GPU), and the wrappers name what is wrong."""
import ctypes

import pytest
import torch

import chunked_gated_delta_amd as kda
from chunked_gated_delta_amd import _lib
from chunked_gated_delta_amd._lib import KdaGdr, KdaGdrGrads, KdaNorm, KdaNormGrads, KdaStride

lib = _lib.load()
ST = 1 << 40
P = [0x7F0000000000 + i * ST for i in range(20)]   # aligned addresses that validation never follows
INVALID = ctypes.c_size_t(-1).value


def dense(B, H, T, D):
    return KdaStride(H * T * D, T * D, D)


def desc(B=1, Hk=1, Hv=2, T=100, dk=64, dv=32, n_seq=0, dtype=1, gate=0, g_min=-5.0, scale=1.0, **st):
    s = dict(q=dense(B, Hk, T, dk), k=dense(B, Hk, T, dk), v=dense(B, Hv, T, dv), w=dense(B, Hv, T, 1), beta=dense(B, Hv, T, 1))
    s.update(st)
    return KdaGdr(B, Hk, Hv, T, dk, dv, n_seq, dtype, gate, g_min, scale, s["q"], s["k"], s["v"], s["w"], s["beta"])


def fwd(d=None, so=None, ws_bytes=1 << 30, **over):
    d = desc() if d is None else d
    a = dict(q=P[0], k=P[1], v=P[2], w=P[3], beta=P[4], S0=None, seq=None, o=P[5], Sf=P[6], ws=P[7])
    a.update(over)
    so = dense(d.B, d.Hv, d.T, d.dv) if so is None else so
    return lib.kda_gdr_chunk_fwd(a["q"], a["k"], a["v"], a["w"], a["beta"], a["S0"], a["seq"], ctypes.byref(d), a["o"], ctypes.byref(so), a["Sf"],
                                 a["ws"], ws_bytes, None)


def bwd(d=None, ws_bytes=1 << 30, sdo=None, strides=None, **over):
    d = desc() if d is None else d
    a = dict(q=P[0], k=P[1], v=P[2], w=P[3], beta=P[4], S0=None, seq=None, dO=P[5], dSf=None, dq=P[6], dk=P[7], dv=P[8], dw=P[9], dbeta=P[10], dS0=P[11], ws=P[12])
    a.update(over)
    k, v, s = dense(d.B, d.Hk, d.T, d.dk), dense(d.B, d.Hv, d.T, d.dv), dense(d.B, d.Hv, d.T, 1)
    g = KdaGdrGrads(a["dq"], a["dk"], a["dv"], a["dw"], a["dbeta"], a["dS0"], *(strides or (k, k, v, s, s)))
    return lib.kda_gdr_chunk_bwd(a["q"], a["k"], a["v"], a["w"], a["beta"], a["S0"], a["seq"], ctypes.byref(d), a["dO"], ctypes.byref(sdo or v), a["dSf"],
                                 ctypes.byref(g), a["ws"], ws_bytes, None)


def step(d=None, n_slots=8, **over):
    d = desc(T=1) if d is None else d
    a = dict(q=P[0], k=P[1], v=P[2], w=P[3], beta=P[4], S=P[5], slots=P[6], o=P[7])
    a.update(over)
    so = dense(d.B, d.Hv, d.T, d.dv)
    return lib.kda_gdr_decode(a["q"], a["k"], a["v"], a["w"], a["beta"], a["S"], n_slots, a["slots"], ctypes.byref(d), a["o"], ctypes.byref(so), None)


@pytest.mark.parametrize("call", [fwd, bwd, step])
@pytest.mark.parametrize("kw,code", [
    (dict(B=0), -2), (dict(Hk=0), -2), (dict(Hv=3, Hk=2), -2), (dict(T=-1), -2), (dict(T=1 << 31), -2), (dict(dk=0), -2), (dict(B=1 << 32), -2),
    (dict(B=1 << 20, T=1 << 20), -2), (dict(B=1 << 24, T=1), -2), (dict(dk=48), -3), (dict(dv=256), -3), (dict(dtype=2), -3), (dict(gate=3), -3),
    (dict(gate=-1), -3), (dict(g_min=0.5), -4), (dict(g_min=float("nan")), -4), (dict(g_min=-float("inf")), -4), (dict(scale=float("inf")), -4),
    (dict(n_seq=2), -2), (dict(q=KdaStride(6400, 6400, 65)), -4), (dict(v=KdaStride(6400, 3200, -32)), -4), (dict(w=KdaStride(0, -1, 1)), -4),
    (dict(T=2, k=KdaStride(128, 128, 1 << 47)), -4)], ids=str)
def test_descriptors(call, kw, code):
    assert call(desc(**({"T": 100} | kw))) == code


@pytest.mark.parametrize("call", [fwd, bwd, step])
@pytest.mark.parametrize("name,dtype,stride", [("q", 1, (1 << 24) + 8), ("k", 0, (1 << 23) + 4), ("v", 1, (1 << 24) + 8), ("w", 1, (1 << 24) + 1)])
def test_token_strides_within_32_bits_a_chunk(call, name, dtype, stride):
    """The kernels address the 64 tokens of a chunk by 32-bit offsets: a token stride past 32 MiB is refused."""
    assert call(desc(T=2, dtype=dtype, **{name: KdaStride(stride, stride, stride)})) == -4


@pytest.mark.parametrize("call,names", [(fwd, ("q", "k", "v", "w", "beta", "o", "ws")), (step, ("q", "k", "v", "w", "beta", "S", "o")),
                                        (bwd, ("q", "k", "v", "w", "beta", "dO", "dq", "dk", "dv", "dw", "dbeta", "ws"))])
def test_null_and_misaligned_pointers(call, names):
    for n in names:
        assert call(**{n: None}) == (-4 if n == "ws" else -1), n
        at = {"q": 0, "k": 1, "v": 2, "w": 3, "beta": 4}.get(n)
        assert call(**{n: (P[at] if at is not None else P[13]) + 1}) == -4, n
    assert lib.kda_gdr_workspace_bytes(None, 0) == INVALID


def test_outputs_apart():
    assert fwd(o=P[2] + 32) == -4                     # inside v
    assert fwd(Sf=P[7]) == -4                         # the workspace
    assert fwd(S0=P[6] + 64) == -4                    # S_final is S0 or apart from it
    assert fwd(S0=P[5]) == -4
    assert bwd(dq=P[0]) == -4 and bwd(dw=P[10]) == -4 and bwd(dS0=P[11], dSf=P[11]) == -4
    assert step(S=P[2]) == -4 and step(o=P[5]) == -4 and step(slots=P[5]) == -4
    # outputs that hold one place twice
    assert fwd(so=KdaStride(6400, 0, 32)) == -4 and fwd(so=KdaStride(6400, 3200, 16)) == -4
    d = desc()
    k, v, s = dense(1, 1, 100, 64), dense(1, 2, 100, 32), dense(1, 2, 100, 1)
    assert bwd(strides=(KdaStride(0, 0, 32), k, v, s, s)) == -4 and bwd(strides=(k, k, v, KdaStride(200, 100, 0), s)) == -4
    assert bwd(d, strides=(k, k, v, s, KdaStride(200, 50, 1))) == -4


def test_workspace_sizes():
    n = lib.kda_gdr_workspace_bytes(ctypes.byref(desc()), 0)
    b = lib.kda_gdr_workspace_bytes(ctypes.byref(desc()), 1)
    assert 0 < n < b < 1 << 30
    assert fwd(ws_bytes=n - 1) == -4 and bwd(ws_bytes=b - 1) == -4
    assert lib.kda_gdr_workspace_bytes(ctypes.byref(desc(T=0)), 1) == 0
    assert lib.kda_gdr_workspace_bytes(ctypes.byref(desc(dk=40)), 0) == INVALID
    assert kda.gdr_workspace_bytes(1, 1, 2, 100, 64, 32) == n and kda.gdr_workspace_bytes(1, 1, 2, 100, 64, 32, backward=True) == b
    # packed sequences: room for each one's last chunk
    assert kda.gdr_workspace_bytes(1, 1, 2, 100, 64, 32, n_seq=5) > n
    with pytest.raises(kda.KdaError):
        kda.gdr_workspace_bytes(2, 1, 2, 100, 64, 32, n_seq=5)


def test_packed_and_pools():
    assert fwd(desc(n_seq=0), seq=P[14]) == -2        # offsets need n_seq
    assert fwd(desc(B=2, n_seq=2), seq=P[14]) == -2
    assert fwd(desc(n_seq=2), seq=P[14] + 2) == -4
    assert step(desc(B=4, T=1), n_slots=3, slots=None) == -2 and step(n_slots=-1) == -2
    assert step(desc(T=0), q=None, k=None, v=None, w=None, beta=None, o=None) == 0


def norm_desc(B=1, H=1, T=4, D=64, dtype=1, wdtype=0, act=1, alpha=1.0, eps=1e-6, **st):
    s = dict(x=dense(B, H, T, D), z=dense(B, H, T, D), residual=dense(B, H, T, D)) | st
    return KdaNorm(B, H, T, D, dtype, wdtype, act, alpha, eps, s["x"], s["z"], s["residual"])


def nfwd(d=None, ss=None, **over):
    d = norm_desc() if d is None else d
    a = dict(x=P[0], weight=P[1], z=P[2], residual=P[3], next_weight=P[4], s=P[5], y=P[6]) | over
    o = dense(d.B, d.H, d.T, d.D)
    return lib.kda_norm_fwd(a["x"], a["weight"], a["z"], a["residual"], a["next_weight"], ctypes.byref(d), a["s"], ctypes.byref(ss or o), a["y"], ctypes.byref(o), None)


def nbwd(d=None, ws_bytes=1 << 30, sx=None, **over):
    d = norm_desc() if d is None else d
    a = dict(x=P[0], weight=P[1], z=P[2], residual=P[3], next_weight=P[4], ds=P[5], dy=P[6], dx=P[7], dz=P[8], dresidual=P[9], dweight=P[10], dnext_weight=P[11],
             ws=P[12]) | over
    o = dense(d.B, d.H, d.T, d.D)
    g = KdaNormGrads(a["dx"], a["dz"], a["dresidual"], a["dweight"], a["dnext_weight"], sx or o, o, o)
    return lib.kda_norm_bwd(a["x"], a["weight"], a["z"], a["residual"], a["next_weight"], ctypes.byref(d), a["ds"], ctypes.byref(o), a["dy"], ctypes.byref(o),
                            ctypes.byref(g), a["ws"], ws_bytes, None)


@pytest.mark.parametrize("call", [nfwd, nbwd])
@pytest.mark.parametrize("kw,code", [(dict(D=0), -2), (dict(B=-1), -2), (dict(D=16385), -3), (dict(T=1 << 40), -2), (dict(dtype=2), -3), (dict(wdtype=5), -3),
                                     (dict(act=2), -3), (dict(alpha=float("nan")), -4), (dict(eps=-1.0), -4), (dict(eps=float("inf")), -4),
                                     (dict(x=KdaStride(0, 0, -64)), -4)], ids=str)
def test_norm_descriptors(call, kw, code):
    assert call(norm_desc(**kw)) == code


def test_norm_pointers():
    for n in ("x", "s", "y"):
        assert nfwd(**{n: None}) == -1, n
    for n in ("x", "dx", "dz", "dresidual", "dweight", "dnext_weight", "dy"):
        assert nbwd(**{n: None}) == -1, n
    assert nbwd(next_weight=None, ds=None) == -1
    assert nfwd(weight=None, next_weight=None) == -4 and nbwd(weight=None, next_weight=None) == -4
    assert nfwd(x=P[0] + 1) == -4 and nfwd(weight=P[1] + 2) == -4 and nbwd(dz=P[8] + 1) == -4
    assert nfwd(s=P[0]) == -4 and nfwd(y=P[5]) == -4 and nbwd(dx=P[5]) == -4 and nbwd(ws=P[7]) == -4
    assert nfwd(ss=KdaStride(256, 256, 0)) == -4 and nbwd(sx=KdaStride(256, 256, 32)) == -4
    assert nbwd(ws=None) == -4 and nbwd(ws_bytes=lib.kda_norm_bwd_workspace_bytes(ctypes.byref(norm_desc())) - 1) == -4
    assert lib.kda_norm_bwd_workspace_bytes(ctypes.byref(norm_desc(D=0))) == INVALID
    assert nfwd(norm_desc(T=0)) == 0                  # no rows: nothing to do


def test_wrappers_name_what_is_wrong():
    x = torch.zeros(1, 1, 4, 32)
    with pytest.raises(ValueError, match="GPU"):
        kda.gdr_chunk_fwd(x, x, x, x[..., 0], x[..., 0])
    with pytest.raises(ValueError, match="GPU"):
        kda.gdr_decode(x, x, x, x[..., 0], x[..., 0], torch.zeros(1, 1, 32, 32))
    with pytest.raises(ValueError, match="GPU"):
        kda.norm_gate_fwd(x, torch.ones(32))
    with pytest.raises(TypeError):
        kda.gdr_workspace_bytes(1, 1, 1, 4, 32, 32, dtype=torch.float16)
    m = torch.zeros(1, 1, 4, 32, device="meta")
    with pytest.raises(ValueError, match="GPU"):
        kda.norm_gate_bwd(m, m, weight=torch.ones(32))
