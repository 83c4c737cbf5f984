"""Refusals of linear attention with a decay for each head and of the norms of queries and keys with rotation, on the
host: every invalid call returns its code before any HIP call (so these run without a GPU), and the wrappers name what is
wrong."""
import ctypes

import pytest
import torch

import chunked_gated_delta_amd as kda
from chunked_gated_delta_amd import _lib
from chunked_gated_delta_amd._lib import KdaLad, KdaLadGrads, KdaQkNorm, KdaQkNormGrads, KdaStride

lib = _lib.load()
ST = 1 << 40
P = [0x7F0000000000 + i * ST for i in range(20)]   # aligned addresses that validation never follows
INVALID = ctypes.c_size_t(-1).value


def dense(B, H, T, D):
    return KdaStride(H * T * D, T * D, D)


def desc(B=1, Hk=1, Hv=2, T=100, dk=64, dv=32, n_seq=0, dtype=1, gate=0, w_per_head=0, g_min=-5.0, scale=1.0, **st):
    s = dict(q=dense(B, Hk, T, dk), k=dense(B, Hk, T, dk), v=dense(B, Hv, T, dv), w=dense(B, Hv, T, 1))
    s.update(st)
    return KdaLad(B, Hk, Hv, T, dk, dv, n_seq, dtype, gate, w_per_head, g_min, scale, s["q"], s["k"], s["v"], s["w"])


def fwd(d=None, so=None, ws_bytes=1 << 40, **over):
    d = desc() if d is None else d
    a = dict(q=P[0], k=P[1], v=P[2], w=P[3], S0=None, seq=None, o=P[5], Sf=P[6], ws=P[7])
    a.update(over)
    so = dense(d.B, d.Hv, d.T, d.dv) if so is None else so
    return lib.kda_lad_chunk_fwd(a["q"], a["k"], a["v"], a["w"], a["S0"], a["seq"], ctypes.byref(d), a["o"], ctypes.byref(so), a["Sf"], a["ws"],
                                 ws_bytes, None)


def bwd(d=None, ws_bytes=1 << 40, sdo=None, strides=None, **over):
    d = desc() if d is None else d
    a = dict(q=P[0], k=P[1], v=P[2], w=P[3], S0=None, seq=None, dO=P[5], dSf=None, dq=P[6], dk=P[7], dv=P[8], dw=P[9], dS0=P[11], ws=P[12])
    a.update(over)
    k, v, s = dense(d.B, d.Hk, d.T, d.dk), dense(d.B, d.Hv, d.T, d.dv), dense(d.B, d.Hv, d.T, 1)
    g = KdaLadGrads(a["dq"], a["dk"], a["dv"], a["dw"], a["dS0"], *(strides or (k, k, v, s)))
    return lib.kda_lad_chunk_bwd(a["q"], a["k"], a["v"], a["w"], a["S0"], a["seq"], ctypes.byref(d), a["dO"], ctypes.byref(sdo or v), a["dSf"],
                                 ctypes.byref(g), a["ws"], ws_bytes, None)


def step(d=None, n_slots=8, **over):
    d = desc(T=1) if d is None else d
    a = dict(q=P[0], k=P[1], v=P[2], w=P[3], S=P[5], slots=P[6], o=P[7])
    a.update(over)
    so = dense(d.B, d.Hv, d.T, d.dv)
    return lib.kda_lad_decode(a["q"], a["k"], a["v"], a["w"], a["S"], n_slots, a["slots"], ctypes.byref(d), a["o"], ctypes.byref(so), None)


@pytest.mark.parametrize("call", [fwd, bwd, step])
@pytest.mark.parametrize("kw,code", [
    (dict(B=0), -2), (dict(Hk=0), -2), (dict(Hv=3, Hk=2), -2), (dict(T=-1), -2), (dict(T=1 << 31), -2), (dict(dk=0), -2), (dict(B=1 << 32), -2),
    (dict(B=1 << 24, T=1), -2), (dict(Hv=1 << 17), -2), (dict(dk=48), -3), (dict(dv=256), -3), (dict(dtype=2), -3), (dict(gate=3), -3),
    (dict(gate=-1), -3), (dict(g_min=0.5), -4), (dict(g_min=float("nan")), -4), (dict(g_min=-float("inf")), -4), (dict(scale=float("inf")), -4),
    (dict(w_per_head=2), -4), (dict(w_per_head=-1), -4), (dict(n_seq=2), -2), (dict(q=KdaStride(6400, 6400, 65)), -4),
    (dict(v=KdaStride(6400, 3200, -32), T=100), -4), (dict(w=KdaStride(0, -1, 1)), -4)])
def test_descriptors(call, kw, code):
    d = dict(T=1) if call is step and "T" not in kw and "v" not in kw and "q" not in kw else {}
    assert call(desc(**{**d, **kw})) == code


@pytest.mark.parametrize("call,names", [(fwd, ("q", "k", "v", "w", "o")), (bwd, ("q", "k", "v", "w", "dO", "dq", "dk", "dv")), (step, ("q", "k", "v", "w", "S", "o"))])
def test_null_pointers(call, names):
    for n in names:
        assert call(**{n: None}) == -1, n


def test_null_structures():
    d, so = desc(), dense(1, 2, 100, 32)
    assert lib.kda_lad_chunk_fwd(P[0], P[1], P[2], P[3], None, None, None, P[5], ctypes.byref(so), P[6], P[7], 1 << 40, None) == -1
    assert lib.kda_lad_chunk_fwd(P[0], P[1], P[2], P[3], None, None, ctypes.byref(d), P[5], None, P[6], P[7], 1 << 40, None) == -1
    assert lib.kda_lad_chunk_bwd(P[0], P[1], P[2], P[3], None, None, ctypes.byref(d), P[5], ctypes.byref(so), None, None, P[7], 1 << 40, None) == -1
    assert lib.kda_lad_workspace_bytes(None, 0) == INVALID


def test_strides_and_alignment():
    big = KdaStride(0, 0, 1 << 25)   # 64 MiB between tokens of bf16
    for call in (fwd, bwd):
        assert call(desc(k=big)) == -4
        assert call(q=P[0] + 8) == -4
        assert call(w=P[3] + 1) == -4
        assert call(S0=P[15] + 4) == -4
        assert call(ws=P[7] + 8) == -4
    assert fwd(so=KdaStride(6400, 3200, 16)) == -4           # rows on one another
    assert fwd(so=KdaStride(6400, 0, 32)) == -4              # heads on one another
    assert fwd(o=P[5] + 2) == -4
    k, v, s = dense(1, 1, 100, 64), dense(1, 2, 100, 32), dense(1, 2, 100, 1)
    assert bwd(strides=(KdaStride(0, 0, 0), k, v, s)) == -4
    assert bwd(strides=(k, k, v, KdaStride(0, 0, 0))) == -4
    assert fwd(desc(w_per_head=1), w=P[3] + 2) == -4
    assert bwd(desc(w_per_head=1), dw=P[9] + 2) == -4
    assert step(S=P[5] + 8) == -4 and step(slots=P[6] + 2) == -4


def test_overlaps():
    assert fwd(o=P[2]) == -4 and fwd(Sf=P[0] + 64) == -4 and fwd(Sf=P[5]) == -4
    assert fwd(S0=P[6] + 16) == -4                                    # S_final partly over S0
    assert bwd(dq=P[0]) == -4 and bwd(dk=P[6]) == -4 and bwd(dw=P[3]) == -4 and bwd(dS0=P[12] + 256) == -4 and bwd(dSf=P[11]) == -4
    assert bwd(desc(w_per_head=1), dw=P[3]) == -4
    assert step(o=P[0]) == -4 and step(S=P[7]) == -4


def test_workspace():
    for bw in (0, 1):
        assert lib.kda_lad_workspace_bytes(ctypes.byref(desc(dk=48)), bw) == INVALID
        assert lib.kda_lad_workspace_bytes(ctypes.byref(desc(n_seq=3, B=2)), bw) == INVALID
    assert lib.kda_lad_workspace_bytes(ctypes.byref(desc(T=100)), 0) == 0
    n = lib.kda_lad_workspace_bytes(ctypes.byref(desc(T=1000)), 0)
    assert 0 < n < 1 << 24
    assert fwd(desc(T=1000), ws=None) == -4 and fwd(desc(T=1000), ws_bytes=n - 1) == -4
    n = lib.kda_lad_workspace_bytes(ctypes.byref(desc()), 1)
    assert 0 < n < 1 << 24
    assert bwd(ws=None) == -4 and bwd(ws_bytes=n - 1) == -4
    assert kda.lad_workspace_bytes(1, 1, 2, 1000, 64, 32) == lib.kda_lad_workspace_bytes(ctypes.byref(desc(T=1000)), 0)
    assert kda.lad_workspace_bytes(1, 1, 2, 1000, 64, 32, n_seq=5, backward=True) > 0
    with pytest.raises(TypeError):
        kda.lad_workspace_bytes(1, 1, 2, 1000, 64, 32, torch.float16)
    with pytest.raises(kda.KdaError):
        kda.lad_workspace_bytes(1, 2, 3, 1000, 64, 32)


@pytest.mark.parametrize("B,T,Hv,n_seq", [(1, 1, 1, 0), (1, 1 << 20, 16, 0), (64, 8192, 64, 0), (1, 1 << 20, 1, 1000), (1, 300, 512, 7), (512, 64, 64, 0), (1, (1 << 31) - 1, 1, 0)])
def test_workspace_holds_every_segment(B, T, Hv, n_seq):
    """The sizes that the library asks for grow with the segments, not with the tokens' states: at most two states a chunk."""
    n = lib.kda_lad_workspace_bytes(ctypes.byref(desc(B=B, T=T, Hk=Hv, Hv=Hv, dk=128, dv=128, n_seq=n_seq)), 0)
    chunks = B * -(-T // 64) + n_seq
    assert n != INVALID and n <= chunks * Hv * (128 * 128 * 4 + 4) + 1024


def test_step_slots():
    assert step(n_slots=-1) == -2 and step(n_slots=0, slots=None) == -2 and step(desc(B=4, T=1), n_slots=3, slots=None) == -2


# ------------------------------------------------------------------------------------ norms of queries and keys, rotation


def qdesc(B=2, Hq=3, Hk=1, T=10, D=64, R=32, dtype=1, wdtype=0, norm=1, interleaved=0, wide=0, q_scale=1.0, k_scale=1.0, eps=1e-6, pos_b=10, pos_t=1, **st):
    s = dict(q=dense(B, Hq, T, D), k=dense(B, Hk, T, D))
    s.update(st)
    return KdaQkNorm(B, Hq, Hk, T, D, R, dtype, wdtype, norm, interleaved, wide, q_scale, k_scale, eps, pos_b, pos_t, s["q"], s["k"])


def qfwd(d=None, **over):
    d = qdesc() if d is None else d
    a = dict(q=P[0], k=P[1], qw=P[2], kw=P[3], pos=P[4], freq=P[5], qo=P[6], ko=P[7], sq=dense(d.B, d.Hq, d.T, d.D), sk=dense(d.B, d.Hk, d.T, d.D))
    a.update(over)
    return lib.kda_qk_norm_fwd(a["q"], a["k"], a["qw"], a["kw"], a["pos"], a["freq"], ctypes.byref(d), a["qo"], ctypes.byref(a["sq"]), a["ko"],
                               ctypes.byref(a["sk"]), None)


def qbwd(d=None, ws_bytes=1 << 40, **over):
    d = qdesc() if d is None else d
    sq, sk = dense(d.B, d.Hq, d.T, d.D), dense(d.B, d.Hk, d.T, d.D)
    a = dict(q=P[0], k=P[1], qw=P[2], kw=P[3], pos=P[4], freq=P[5], dqo=P[6], dko=P[7], dq=P[8], dk=P[9], dqw=P[10], dkw=P[11], ws=P[12], sq=sq, sk=sk)
    a.update(over)
    g = KdaQkNormGrads(a["dq"], a["dk"], a["dqw"], a["dkw"], a["sq"], a["sk"])
    return lib.kda_qk_norm_bwd(a["q"], a["k"], a["qw"], a["kw"], a["pos"], a["freq"], ctypes.byref(d), a["dqo"], ctypes.byref(sq), a["dko"],
                               ctypes.byref(sk), ctypes.byref(g), a["ws"], ws_bytes, None)


@pytest.mark.parametrize("call", [qfwd, qbwd])
@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), -2), (dict(T=-1), -2), (dict(Hq=-1), -2), (dict(Hk=1 << 17), -2), (dict(D=0), -2), (dict(D=63, R=2), -2), (dict(R=66), -2), (dict(R=3), -2),
    (dict(R=-2), -2), (dict(D=1026), -3), (dict(B=1 << 30, T=4), -2), (dict(B=1 << 25, T=8), -2), (dict(dtype=2), -3), (dict(wdtype=5), -3), (dict(norm=2), -4),
    (dict(interleaved=-1), -4), (dict(wide=3), -4), (dict(eps=-1.0), -4), (dict(eps=float("inf")), -4), (dict(q_scale=float("nan")), -4),
    (dict(k_scale=float("inf")), -4), (dict(q=KdaStride(-1, 640, 64)), -4), (dict(pos_t=-1), -4), (dict(pos_b=-1), -4)])
def test_qk_descriptors(call, kw, code):
    assert call(qdesc(**kw)) == code


def test_qk_nulls_and_overlaps():
    for n in ("q", "k", "pos", "freq", "qo", "ko"):
        assert qfwd(**{n: None}) == -1, n
    for n in ("q", "k", "pos", "freq", "dqo", "dko", "dq", "dk", "dqw", "dkw"):
        assert qbwd(**{n: None}) == -1, n
    assert lib.kda_qk_norm_bwd_workspace_bytes(None) == INVALID
    n = lib.kda_qk_norm_bwd_workspace_bytes(ctypes.byref(qdesc()))
    assert 0 < n < 1 << 24
    assert qbwd(ws=None) == -4 and qbwd(ws_bytes=n - 1) == -4 and qbwd(ws=P[12] + 4) == -4
    assert qfwd(qo=P[0]) == -4 and qfwd(ko=P[6] + 64) == -4 and qfwd(qo=P[4]) == -4 and qfwd(ko=P[2]) == -4
    assert qbwd(dq=P[6]) == -4 and qbwd(dk=P[8]) == -4 and qbwd(dqw=P[2]) == -4 and qbwd(dkw=P[10]) == -4 and qbwd(dq=P[12]) == -4
    assert qfwd(sq=KdaStride(0, 640, 64)) == -4 and qbwd(sk=KdaStride(640, 0, 32)) == -4
    assert qfwd(q=P[0] + 1) == -4 and qfwd(qw=P[2] + 2) == -4 and qfwd(pos=P[4] + 2) == -4 and qfwd(freq=P[5] + 1) == -4
    assert qfwd(qdesc(wide=1), pos=P[4] + 4) == -4


def test_wrappers_name_what_is_wrong():
    """The wrappers refuse tensors that are not on a GPU before anything else."""
    x, w = torch.zeros(1, 1, 4, 32), torch.zeros(1, 1, 4)
    S = torch.zeros(1, 1, 32, 32)
    for call in (lambda: kda.lad_chunk_fwd(x, x, x, w), lambda: kda.lad_chunk_bwd(x, x, x, w, x), lambda: kda.lad_decode(x, x, x, w, S),
                 lambda: kda.qk_norm_rope_fwd(x, x), lambda: kda.qk_norm_rope_bwd(x, x, x, x)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(TypeError, match="q must be a torch tensor"):
        kda.lad_chunk_fwd(None, x, x, w)
    with pytest.raises(TypeError, match="q must be a torch tensor"):
        kda.qk_norm_rope_fwd(None, x)
