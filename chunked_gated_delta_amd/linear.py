"""torch-facing wrappers of linear attention with a decay for each head, and of the norms of queries and keys with
their rotation by position.  Argument marshalling only, as in gated.py, whose rules on strides and streams hold here:
tensors may be strided views with a contiguous last dimension, nothing is copied, and a call with `stream` reads its
inputs there.  The rows of lad's q, k, v, o and dO lie on 16-byte places with tokens at most 32 MiB apart; those of the
norms may lie anywhere."""
from __future__ import annotations

import ctypes
import math
from functools import partial

import torch

from . import _lib
from ._lib import KdaError, KdaLad, KdaLadGrads, KdaQkNorm, KdaQkNormGrads, KdaStride
from .api import _dtype_code, _on_stream
from .gated import _at, _call, _dense, _gpu, _like, _sequences, _view, _workspace

_NONE = KdaStride(0, 0, 0)
_NO_SIZE = ctypes.c_size_t(-1).value


def _stream(dev):
    """The handle of the device's current stream; the Stream object around it costs a microsecond."""
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _out(given, like, name, dev):
    """The output and its strides: the one given, checked, or a new one in the input's order of dimensions."""
    if given is not None:
        return given, _view(given, name, like.shape, like.dtype, dev)
    t = _like(like)
    st = t.stride()
    return t, KdaStride(st[0], st[1], st[2])


def _rows(q, name):
    st = q.stride()
    if st[3] != 1 and q.shape[3] > 1:
        raise ValueError(f"{name} must have a contiguous last dimension")
    return KdaStride(st[0], st[1], st[2])


def _describe(q, k, v, w, g_min, scale, log_decay, n_seq):
    """Checks the inputs; their descriptor."""
    dev = _gpu(q, "q")
    if q.dim() != 4:
        raise ValueError("q must be [B,Hk,T,dk]")
    if not isinstance(v, torch.Tensor) or v.dim() != 4:
        raise ValueError("v must be a [B,Hv,T,dv] tensor")
    B, Hk, T, dk = q.shape
    Hv, dv = v.shape[1], v.shape[3]
    dt = q.dtype
    code = _dtype_code(q)
    sq = _rows(q, "q")
    sk = _view(k, "k", q.shape, dt, dev)
    sv = _view(v, "v", (B, Hv, T, dv), dt, dev)
    per_head = isinstance(w, torch.Tensor) and w.dim() == 1
    if per_head:
        _dense(w, "w", (Hv,), torch.float32, dev)
        sw = _NONE
    else:
        sw = _view(w, "w", (B, Hv, T), dt, dev, rows=False)
    gate = 2 if log_decay else 1 if g_min == -math.inf else 0
    return KdaLad(B, Hk, Hv, T, dk, dv, n_seq, code, gate, per_head, g_min if gate == 0 else 0.0, scale, sq, sk, sv, sw), dev


def _need(desc, backward):
    n = _lib.load().kda_lad_workspace_bytes(ctypes.byref(desc), int(backward))
    return 0 if n == _NO_SIZE else n   # an invalid descriptor: the call itself reports it


def lad_workspace_bytes(B, Hk, Hv, T, dk, dv, dtype=torch.bfloat16, n_seq: int = 0, backward: bool = False) -> int:
    """Scratch of lad_chunk_fwd (or lad_chunk_bwd) for a shape; n_seq: the packed sequences, 0 if not packed."""
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"unsupported dtype {dtype}: use torch.bfloat16 or torch.float32")
    desc = KdaLad(B, Hk, Hv, T, dk, dv, n_seq, 1 if dtype == torch.bfloat16 else 0, 2, 0, 0.0, 1.0, _NONE, _NONE, _NONE, _NONE)
    n = _lib.load().kda_lad_workspace_bytes(ctypes.byref(desc), int(backward))
    if n == _NO_SIZE:
        raise KdaError(_lib.KDA_ERR_SHAPE, "kda_lad_workspace_bytes")
    return n


def lad_chunk_fwd(q, k, v, w, S0=None, g_min: float = -5.0, *, scale: float = 1.0, log_decay: bool = False, cu_seqlens=None,
                  out=None, S_final=None, workspace=None, stream=None):
    """Linear attention with a decay for each head, chunked, through kda_lad_chunk_fwd: (o, S_final).

        S <- e^g S + k v^T;  o = scale S^T q

    q, k: [B,Hk,T,dk]; v: [B,Hv,T,dv] (bf16 or fp32, on one GPU, strided views with a contiguous last dimension); Hk
    divides Hv and value head h uses query/key head h // (Hv // Hk); dk, dv in {32, 64, 128}.  w gives the log-decay
    g: g_min * sigmoid(w), -softplus(w) for g_min = -inf, or w itself (<= 0) with log_decay; it is [B,Hv,T] of the
    inputs' type, or [Hv] in fp32 for one decay a head.  `cu_seqlens` (int32 [n + 1], on the GPU, with B = 1) divides T
    into packed sequences; tokens behind the last one are left as they were (undefined in an output that is allocated
    here).  S0, S_final: fp32 [sequences,Hv,dk,dv]; S_final may be S0 itself.  Asynchronous on `stream` (default: the
    current torch stream)."""
    if stream is not None:
        call = partial(lad_chunk_fwd, q, k, v, w, S0, g_min, scale=scale, log_decay=log_decay, cu_seqlens=cu_seqlens, out=out,
                       S_final=S_final, workspace=workspace)
        return _on_stream(stream, call, q, k, v, w, S0, cu_seqlens, workspace)
    n_seq = _sequences(cu_seqlens, q.device if isinstance(q, torch.Tensor) else None)
    desc, dev = _describe(q, k, v, w, g_min, scale, log_decay, n_seq)
    states = (n_seq or desc.B, desc.Hv, desc.dk, desc.dv)
    if S0 is not None:
        _dense(S0, "S0", states, torch.float32, dev)
    out, so = _out(out, v, "out", dev)
    if S_final is None:
        S_final = torch.empty(states, dtype=torch.float32, device=dev)
    else:
        _dense(S_final, "S_final", states, torch.float32, dev)
    need = _need(desc, False)
    workspace = _workspace(workspace, need, dev)
    _call("kda_lad_chunk_fwd", dev, (_at(q), _at(k), _at(v), _at(w), _at(S0), _at(cu_seqlens), ctypes.byref(desc), _at(out), ctypes.byref(so),
                                     _at(S_final), _at(workspace), need, _stream(dev)))
    return out, S_final


def lad_chunk_bwd(q, k, v, w, dO, S0=None, dS_final=None, g_min: float = -5.0, *, scale: float = 1.0, log_decay: bool = False,
                  cu_seqlens=None, want_dw: bool = True, want_dS0: bool = True, workspace=None, stream=None):
    """Gradients of lad_chunk_fwd through kda_lad_chunk_bwd, given dO = dL/do [B,Hv,T,dv] (the inputs' type) and dS_final
    = dL/dS_final (fp32, None for zero): (dq, dk, dv, dw, dS0), each of its input's shape and type, dS0 fp32 (dw and
    dS0 None where they are not wanted).  The gradient of a broadcast input comes at the broadcast shape; tokens of no
    sequence are left undefined.  Asynchronous on `stream`."""
    if stream is not None:
        call = partial(lad_chunk_bwd, q, k, v, w, dO, S0, dS_final, g_min, scale=scale, log_decay=log_decay, cu_seqlens=cu_seqlens,
                       want_dw=want_dw, want_dS0=want_dS0, workspace=workspace)
        return _on_stream(stream, call, q, k, v, w, dO, S0, dS_final, cu_seqlens, workspace)
    n_seq = _sequences(cu_seqlens, q.device if isinstance(q, torch.Tensor) else None)
    desc, dev = _describe(q, k, v, w, g_min, scale, log_decay, n_seq)
    states = (n_seq or desc.B, desc.Hv, desc.dk, desc.dv)
    sdo = _view(dO, "dO", v.shape, v.dtype, dev)
    if S0 is not None:
        _dense(S0, "S0", states, torch.float32, dev)
    if dS_final is not None:
        _dense(dS_final, "dS_final", states, torch.float32, dev)
    dq, dk, dv = _like(q), _like(k), _like(v)
    dw = _like(w, rows=False) if want_dw else None
    dS0 = torch.empty(states, dtype=torch.float32, device=dev) if want_dS0 else None
    need = _need(desc, True)
    workspace = _workspace(workspace, need, dev)
    at = lambda t: _NONE if t is None or t.dim() == 1 else KdaStride(*t.stride()[:3])  # noqa: E731
    grads = KdaLadGrads(_at(dq), _at(dk), _at(dv), _at(dw), _at(dS0), at(dq), at(dk), at(dv), at(dw))
    _call("kda_lad_chunk_bwd", dev, (_at(q), _at(k), _at(v), _at(w), _at(S0), _at(cu_seqlens), ctypes.byref(desc), _at(dO), ctypes.byref(sdo),
                                     _at(dS_final), ctypes.byref(grads), _at(workspace), need, _stream(dev)))
    return dq, dk, dv, dw, dS0


def lad_decode(q, k, v, w, S, slots=None, g_min: float = -5.0, *, scale: float = 1.0, log_decay: bool = False, out=None, stream=None):
    """Recurrent step through kda_lad_decode: advances states of the pool S (fp32 [n_slots,Hv,dk,dv]) in place by the T
    tokens of each row of q, k [B,Hk,T,dk], v [B,Hv,T,dv], w ([B,Hv,T], or [Hv] in fp32) and returns o.  `slots`
    (int32 [B], on the GPU) names each row's state (None: row b has state b); a row with a slot outside the pool (-1,
    say) is padding and gets zeros; rows with the same slot are that state's successive tokens, in row order.
    Asynchronous on `stream` (default: the current torch stream)."""
    if stream is not None:
        call = partial(lad_decode, q, k, v, w, S, slots, g_min, scale=scale, log_decay=log_decay, out=out)
        return _on_stream(stream, call, q, k, v, w, S, slots)
    desc, dev = _describe(q, k, v, w, g_min, scale, log_decay, 0)
    if not isinstance(S, torch.Tensor) or S.dim() != 4:
        raise ValueError("S must be a [n_slots,Hv,dk,dv] tensor")
    _dense(S, "S", (S.shape[0], desc.Hv, desc.dk, desc.dv), torch.float32, dev)
    if slots is not None:
        _dense(slots, "slots", (desc.B,), torch.int32, dev)
    elif S.shape[0] < desc.B:
        raise ValueError(f"S has {S.shape[0]} states for {desc.B} rows")
    out, so = _out(out, v, "out", dev)
    _call("kda_lad_decode", dev, (_at(q), _at(k), _at(v), _at(w), _at(S), S.shape[0], _at(slots), ctypes.byref(desc), _at(out), ctypes.byref(so),
                                  _stream(dev)))
    return out


# ------------------------------------------------------------------------------------ norms of queries and keys, rotation


def _qk_describe(q, k, q_weight, k_weight, positions, inv_freq, norm, interleaved, q_scale, k_scale, eps):
    dev = _gpu(q, "q")
    if q.dim() != 4:
        raise ValueError("q must be [B,Hq,T,D]")
    B, Hq, T, D = q.shape
    code = _dtype_code(q)
    sq, sk, Hk = _rows(q, "q"), _NONE, 0
    if k is not None:
        if not isinstance(k, torch.Tensor) or k.dim() != 4:
            raise ValueError("k must be a [B,Hk,T,D] tensor")
        Hk = k.shape[1]
        sk = _view(k, "k", (B, Hk, T, D), q.dtype, dev)
    elif k_weight is not None:
        raise ValueError("k_weight is given without k")
    wcode = code
    lead = q_weight if q_weight is not None else k_weight
    if lead is not None:
        if not isinstance(lead, torch.Tensor):
            raise TypeError("weights must be torch tensors")
        wcode = _dtype_code(lead)
        for t, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
            if t is not None:
                _dense(t, name, (D,), lead.dtype, dev)
    if (positions is None) != (inv_freq is None):
        raise ValueError("positions and inv_freq are given together or not at all")
    if not norm and lead is None and inv_freq is None:
        raise ValueError("norm is False and there are neither weights nor a rotation: nothing to do")
    R, wide, pos = 0, False, (0, 0)
    if inv_freq is not None:
        if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
            raise ValueError("inv_freq must be a tensor of the pairs' frequencies")
        _dense(inv_freq, "inv_freq", inv_freq.shape, torch.float32, dev)
        R = 2 * inv_freq.shape[0]
        if R > D:
            raise ValueError(f"inv_freq has {inv_freq.shape[0]} frequencies for rows of {D}")
        if not isinstance(positions, torch.Tensor):
            raise TypeError("positions must be a torch tensor")
        if positions.dtype not in (torch.int32, torch.int64):
            raise TypeError(f"positions has dtype {positions.dtype}, expected torch.int32 or torch.int64")
        if positions.device != dev:
            raise ValueError(f"positions is on {positions.device}, expected {dev}")
        if positions.shape != (B, T) and positions.shape != (T,):
            raise ValueError(f"positions has shape {tuple(positions.shape)}, expected {(B, T)} or {(T,)}")
        wide = positions.dtype == torch.int64
        pos = positions.stride() if positions.dim() == 2 else (0, positions.stride(0))
    return KdaQkNorm(B, Hq, Hk, T, D, R, code, wcode, bool(norm), bool(interleaved), wide, q_scale, k_scale, eps, pos[0], pos[1], sq, sk), dev


def qk_norm_rope_fwd(q, k, q_weight=None, k_weight=None, positions=None, inv_freq=None, *, norm: bool = True, interleaved: bool = False,
                     q_scale: float = 1.0, k_scale: float = 1.0, eps: float = 1e-6, q_out=None, k_out=None, stream=None):
    """Norms of queries and keys for each head and their rotation by position, through kda_qk_norm_fwd: (q_out, k_out).

        n = x / rms(x) * weight;  y = scale * n, its first values rotated in pairs by the angles position * inv_freq

    q: [B,Hq,T,D]; k: [B,Hk,T,D] or None (bf16 or fp32, any strides with a contiguous last dimension; D even, up to
    1024).  norm False leaves out the division, a weight of None the product; weights [D], both bf16 or both fp32.
    positions: int32 or int64, [B,T] or [T]; inv_freq: fp32 [R/2], R <= D: pair i of a row is values i and i + R/2, or 2i
    and 2i + 1 with `interleaved`; both None leave out the rotation.  Angles are formed in 64 bits and rounded once.  Rows of unit
    length, as a delta rule's keys, are those without a weight at a scale of D ** -0.5.  Outputs lie apart from every
    input (nothing is done in place).  Asynchronous on `stream`."""
    if stream is not None:
        call = partial(qk_norm_rope_fwd, q, k, q_weight, k_weight, positions, inv_freq, norm=norm, interleaved=interleaved, q_scale=q_scale,
                       k_scale=k_scale, eps=eps, q_out=q_out, k_out=k_out)
        return _on_stream(stream, call, q, k, q_weight, k_weight, positions, inv_freq)
    desc, dev = _qk_describe(q, k, q_weight, k_weight, positions, inv_freq, norm, interleaved, q_scale, k_scale, eps)
    if k is None and k_out is not None:
        raise ValueError("k_out is given without k")
    q_out, sq = _out(q_out, q, "q_out", dev)
    k_out, sk = _out(k_out, k, "k_out", dev) if k is not None else (None, _NONE)
    _call("kda_qk_norm_fwd", dev, (_at(q), _at(k), _at(q_weight), _at(k_weight), _at(positions), _at(inv_freq), ctypes.byref(desc), _at(q_out),
                                   ctypes.byref(sq), _at(k_out), ctypes.byref(sk), _stream(dev)))
    return q_out, k_out


def qk_norm_rope_bwd(q, k, dq_out, dk_out, q_weight=None, k_weight=None, positions=None, inv_freq=None, *, norm: bool = True,
                     interleaved: bool = False, q_scale: float = 1.0, k_scale: float = 1.0, eps: float = 1e-6, workspace=None, stream=None):
    """Gradients of qk_norm_rope_fwd through kda_qk_norm_bwd, given dq_out = dL/dq_out and dk_out = dL/dk_out:
    (dq, dk, dq_weight, dk_weight), None for what was not given; rows' gradients in q's type, weights' in the weights'.
    Asynchronous on `stream`."""
    if stream is not None:
        call = partial(qk_norm_rope_bwd, q, k, dq_out, dk_out, q_weight, k_weight, positions, inv_freq, norm=norm, interleaved=interleaved,
                       q_scale=q_scale, k_scale=k_scale, eps=eps, workspace=workspace)
        return _on_stream(stream, call, q, k, dq_out, dk_out, q_weight, k_weight, positions, inv_freq, workspace)
    desc, dev = _qk_describe(q, k, q_weight, k_weight, positions, inv_freq, norm, interleaved, q_scale, k_scale, eps)
    if (dk_out is None) != (k is None):
        raise ValueError("dk_out is given exactly when k is")
    sdq = _view(dq_out, "dq_out", q.shape, q.dtype, dev)
    sdk = _view(dk_out, "dk_out", k.shape, k.dtype, dev) if k is not None else _NONE
    dq = _like(q)
    dk = _like(k) if k is not None else None
    dqw = torch.empty_like(q_weight) if q_weight is not None else None
    dkw = torch.empty_like(k_weight) if k_weight is not None else None
    need = _lib.load().kda_qk_norm_bwd_workspace_bytes(ctypes.byref(desc)) if dqw is not None or dkw is not None else 0
    need = 0 if need == _NO_SIZE else need
    workspace = _workspace(workspace, need, dev)
    at = lambda t: _NONE if t is None else KdaStride(*t.stride()[:3])  # noqa: E731
    grads = KdaQkNormGrads(_at(dq), _at(dk), _at(dqw), _at(dkw), at(dq), at(dk))
    _call("kda_qk_norm_bwd", dev, (_at(q), _at(k), _at(q_weight), _at(k_weight), _at(positions), _at(inv_freq), ctypes.byref(desc), _at(dq_out),
                                   ctypes.byref(sdq), _at(dk_out), ctypes.byref(sdk), ctypes.byref(grads), _at(workspace), need, _stream(dev)))
    return dq, dk, dqw, dkw
