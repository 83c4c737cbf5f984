"""torch-facing wrappers of the head-gated delta rule (one log-decay per token and head) and of the norms
around a block.  Argument marshalling only, as in api.py: the computation is in the library's HIP kernels.

Tensors may be strided views with a contiguous last dimension, so [B,T,H,D] projections are passed as
x.transpose(1, 2) and slices of a fused projection as they are; nothing is copied.  The rule's q, k, v, o and dO have
their rows on 16-byte places and their tokens at most 32 MiB apart; the norms' rows may lie anywhere.

A call with `stream` reads its inputs there: whoever wrote them on another stream lets `stream` wait for that
one first, and whoever uses the results on another stream lets that one wait for `stream`."""
from __future__ import annotations

import ctypes
import math
from functools import partial

import torch

from . import _lib
from ._lib import KdaError, KdaGdr, KdaGdrGrads, KdaNorm, KdaNormGrads, KdaStride
from .api import _dtype_code, _on_stream

_ACTS = {"sigmoid": 0, "silu": 1}


def _view(t, name, shape, dtype, device, rows=True):
    """Checks one strided tensor; its strides over batch, heads and tokens."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    st = t.stride()
    if rows and st[3] != 1 and shape[3] > 1:
        raise ValueError(f"{name} must have a contiguous last dimension")
    return KdaStride(st[0], st[1], st[2])


def _dense(t, name, shape, dtype, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _at(t):
    return t.data_ptr() if t is not None else None


def _like(t, rows=True):
    """An uninitialised tensor of t's shape, in t's order of dimensions where that keeps rows contiguous."""
    st = t.stride()
    if 0 not in st:
        out = torch.empty_like(t)
        if not rows or out.stride(-1) == 1 or t.shape[-1] == 1:
            return out
    return torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _gpu(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.device.type != "cuda":
        raise ValueError("inputs must live on a GPU (the library has no CPU path)")
    return t.device


def _call(name, dev, args):
    fn = getattr(_lib.load(), name)
    if dev.index == torch.cuda.current_device():   # the guard costs more than a microsecond
        rc = fn(*args)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args)
    if rc != 0:
        raise KdaError(rc, name, _lib.last_hip_error() if rc == _lib.KDA_ERR_HIP else "")


def _describe(q, k, v, w, beta, g_min, scale, log_decay, n_seq):
    """Checks the rule's inputs; their descriptor."""
    dev = _gpu(q, "q")
    if q.dim() != 4:
        raise ValueError("q must be [B,Hk,T,dk]")
    if not isinstance(v, torch.Tensor) or v.dim() != 4:
        raise ValueError("v must be a [B,Hv,T,dv] tensor")
    B, Hk, T, dk = q.shape
    Hv, dv = v.shape[1], v.shape[3]
    dt = q.dtype
    code = _dtype_code(q)
    sq = _view(q, "q", q.shape, dt, dev)
    sk = _view(k, "k", q.shape, dt, dev)
    sv = _view(v, "v", (B, Hv, T, dv), dt, dev)
    sw = _view(w, "w", (B, Hv, T), dt, dev, rows=False)
    sb = _view(beta, "beta", (B, Hv, T), dt, dev, rows=False)
    if log_decay:
        gate = 2
    else:
        gate = 1 if g_min == -math.inf else 0
    return KdaGdr(B, Hk, Hv, T, dk, dv, n_seq, code, gate, g_min if gate == 0 else 0.0, scale, sq, sk, sv, sw, sb), dev


def _sequences(cu_seqlens, dev):
    if cu_seqlens is None:
        return 0
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be a tensor of the sequences' offsets (one more than sequences)")
    _dense(cu_seqlens, "cu_seqlens", cu_seqlens.shape, torch.int32, dev)
    return cu_seqlens.numel() - 1


def _workspace(workspace, need, dev):
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    if not workspace.is_contiguous() or workspace.device != dev:
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    if workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace holds {workspace.numel() * workspace.element_size()} bytes, {need} needed")
    return workspace


def _need(desc, backward):
    n = _lib.load().kda_gdr_workspace_bytes(ctypes.byref(desc), int(backward))
    return 0 if n == ctypes.c_size_t(-1).value else n   # an invalid descriptor: the call itself reports it


def gdr_workspace_bytes(B, Hk, Hv, T, dk, dv, dtype=torch.bfloat16, n_seq: int = 0, backward: bool = False) -> int:
    """Scratch of gdr_chunk_fwd (or gdr_chunk_bwd) for a shape; n_seq: the packed sequences, 0 if not packed."""
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"unsupported dtype {dtype}: use torch.bfloat16 or torch.float32")
    z = KdaStride(0, 0, 0)
    desc = KdaGdr(B, Hk, Hv, T, dk, dv, n_seq, 1 if dtype == torch.bfloat16 else 0, 2, 0.0, 1.0, z, z, z, z, z)
    n = _lib.load().kda_gdr_workspace_bytes(ctypes.byref(desc), int(backward))
    if n == ctypes.c_size_t(-1).value:
        raise KdaError(_lib.KDA_ERR_SHAPE, "kda_gdr_workspace_bytes")
    return n


def gdr_chunk_fwd(q, k, v, w, beta, S0=None, g_min: float = -5.0, *, scale: float = 1.0, log_decay: bool = False,
                  cu_seqlens=None, out=None, S_final=None, workspace=None, stream=None):
    """Head-gated delta rule, chunked, through kda_gdr_chunk_fwd: (o, S_final).

    q, k: [B,Hk,T,dk]; v: [B,Hv,T,dv]; w, beta: [B,Hv,T] (all bf16 or all fp32, on one GPU, strided views
    with a contiguous last dimension of q, k, v); Hk divides Hv and value head h uses query/key head
    h // (Hv // Hk); dk, dv in {32, 64, 128}.  The log-decay is g_min * sigmoid(w), -softplus(w) for
    g_min = -inf, or w itself (<= 0) with log_decay.  `cu_seqlens` (int32 [n + 1], on the GPU, with B = 1)
    divides T into packed sequences; tokens behind the last one are left as they were (undefined in an
    output that is allocated here).  S0, S_final: fp32 [sequences,Hv,dk,dv]; S_final may be S0 itself.
    Asynchronous on `stream` (default: the current torch stream)."""
    if stream is not None:
        call = partial(gdr_chunk_fwd, q, k, v, w, beta, S0, g_min, scale=scale, log_decay=log_decay,
                       cu_seqlens=cu_seqlens, out=out, S_final=S_final, workspace=workspace)
        return _on_stream(stream, call, q, k, v, w, beta, S0, cu_seqlens, workspace)
    n_seq = _sequences(cu_seqlens, q.device if isinstance(q, torch.Tensor) else None)
    desc, dev = _describe(q, k, v, w, beta, g_min, scale, log_decay, n_seq)
    states = (n_seq or desc.B, desc.Hv, desc.dk, desc.dv)
    if S0 is not None:
        _dense(S0, "S0", states, torch.float32, dev)
    if out is None:
        out = _like(v)
    so = _view(out, "out", v.shape, v.dtype, dev)
    if S_final is None:
        S_final = torch.empty(states, dtype=torch.float32, device=dev)
    else:
        _dense(S_final, "S_final", states, torch.float32, dev)
    need = _need(desc, False)
    workspace = _workspace(workspace, need, dev)
    stream = torch.cuda.current_stream(dev.index)
    _call("kda_gdr_chunk_fwd", dev, (_at(q), _at(k), _at(v), _at(w), _at(beta), _at(S0), _at(cu_seqlens), ctypes.byref(desc), _at(out),
                                     ctypes.byref(so), _at(S_final), _at(workspace), need, stream.cuda_stream))
    return out, S_final


def gdr_chunk_bwd(q, k, v, w, beta, dO, S0=None, dS_final=None, g_min: float = -5.0, *, scale: float = 1.0,
                  log_decay: bool = False, cu_seqlens=None, want_dS0: bool = True, workspace=None, stream=None):
    """Gradients of gdr_chunk_fwd through kda_gdr_chunk_bwd, given dO = dL/do [B,Hv,T,dv] (the inputs' type)
    and dS_final = dL/dS_final (fp32, None for zero): (dq, dk, dv, dw, dbeta, dS0), each of its input's shape
    and type, dS0 fp32 (None when want_dS0 is False).  The gradient of a broadcast input comes at the
    broadcast shape; tokens of no sequence are left undefined.  Asynchronous on `stream`."""
    if stream is not None:
        call = partial(gdr_chunk_bwd, q, k, v, w, beta, dO, S0, dS_final, g_min, scale=scale, log_decay=log_decay,
                       cu_seqlens=cu_seqlens, want_dS0=want_dS0, workspace=workspace)
        return _on_stream(stream, call, q, k, v, w, beta, dO, S0, dS_final, cu_seqlens, workspace)
    n_seq = _sequences(cu_seqlens, q.device if isinstance(q, torch.Tensor) else None)
    desc, dev = _describe(q, k, v, w, beta, g_min, scale, log_decay, n_seq)
    states = (n_seq or desc.B, desc.Hv, desc.dk, desc.dv)
    sdo = _view(dO, "dO", v.shape, v.dtype, dev)
    if S0 is not None:
        _dense(S0, "S0", states, torch.float32, dev)
    if dS_final is not None:
        _dense(dS_final, "dS_final", states, torch.float32, dev)
    outs = [_like(q), _like(k), _like(v), _like(w, rows=False), _like(beta, rows=False)]
    dS0 = torch.empty(states, dtype=torch.float32, device=dev) if want_dS0 else None
    need = _need(desc, True)
    workspace = _workspace(workspace, need, dev)
    stream = torch.cuda.current_stream(dev.index)
    grads = KdaGdrGrads(*(_at(t) for t in outs), _at(dS0), *(KdaStride(*t.stride()[:3]) for t in outs))
    _call("kda_gdr_chunk_bwd", dev, (_at(q), _at(k), _at(v), _at(w), _at(beta), _at(S0), _at(cu_seqlens), ctypes.byref(desc), _at(dO),
                                     ctypes.byref(sdo), _at(dS_final), ctypes.byref(grads), _at(workspace), need, stream.cuda_stream))
    return (*outs, dS0)


def gdr_decode(q, k, v, w, beta, S, slots=None, g_min: float = -5.0, *, scale: float = 1.0, log_decay: bool = False,
               out=None, stream=None):
    """Recurrent step through kda_gdr_decode: advances states of the pool S (fp32 [n_slots,Hv,dk,dv]) in place
    by the T tokens of each row of q, k [B,Hk,T,dk], v [B,Hv,T,dv], w, beta [B,Hv,T] and returns o.
    `slots` (int32 [B], on the GPU) names each row's state (None: row b has state b); a row with a slot
    outside the pool (-1, say) is padding and gets zeros; rows with the same slot are that state's
    successive tokens, in row order.  Asynchronous on `stream` (default: the current torch stream)."""
    if stream is not None:
        call = partial(gdr_decode, q, k, v, w, beta, S, slots, g_min, scale=scale, log_decay=log_decay, out=out)
        return _on_stream(stream, call, q, k, v, w, beta, S, slots)
    desc, dev = _describe(q, k, v, w, beta, g_min, scale, log_decay, 0)
    if not isinstance(S, torch.Tensor) or S.dim() != 4:
        raise ValueError("S must be a [n_slots,Hv,dk,dv] tensor")
    _dense(S, "S", (S.shape[0], desc.Hv, desc.dk, desc.dv), torch.float32, dev)
    if slots is not None:
        _dense(slots, "slots", (desc.B,), torch.int32, dev)
    elif S.shape[0] < desc.B:
        raise ValueError(f"S has {S.shape[0]} states for {desc.B} rows")
    if out is None:
        out = _like(v)
    so = _view(out, "out", v.shape, v.dtype, dev)
    stream = torch.cuda.current_stream(dev.index)
    _call("kda_gdr_decode", dev, (_at(q), _at(k), _at(v), _at(w), _at(beta), _at(S), S.shape[0], _at(slots), ctypes.byref(desc), _at(out),
                                  ctypes.byref(so), stream.cuda_stream))
    return out


def _row_strides(t):
    """Strides of a tensor of up to four dimensions over its rows' places [B,H,T] (those it lacks: 0)."""
    return KdaStride(*((0, 0, 0) + t.stride())[-4:-1])


def _rows(t, name, x):
    """Checks a tensor of rows against x; its strides over them."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.shape != x.shape:
        raise ValueError(f"{name} must be a tensor of x's shape {tuple(x.shape)}, not {tuple(t.shape)}")
    if t.dtype != x.dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {x.dtype}")
    if t.device != x.device:
        raise ValueError(f"{name} is on {t.device}, expected {x.device}")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must have a contiguous last dimension")
    return _row_strides(t)


def _norm_inputs(x, weight, z, act, residual, alpha, next_weight, eps):
    dev = _gpu(x, "x")
    if not 1 <= x.dim() <= 4:
        raise ValueError("x must have one to four dimensions")
    if weight is None and next_weight is None:
        raise ValueError("weight and next_weight are both None: nothing to normalise")
    if act not in ("silu", "sigmoid", "none"):
        raise ValueError(f"act is {act!r}: use 'silu', 'sigmoid' or, without z, 'none'")
    if act == "none" and z is not None:
        raise ValueError("z is given with act 'none'")
    code, D = _dtype_code(x), x.shape[-1]
    lead = weight if weight is not None else next_weight
    if not isinstance(lead, torch.Tensor):
        raise TypeError("weights must be torch tensors")
    wcode = _dtype_code(lead)
    for t, name in ((weight, "weight"), (next_weight, "next_weight")):
        if t is not None:
            _dense(t, name, (D,), lead.dtype, dev)
    none = KdaStride(0, 0, 0)
    strides = [none if t is None else _rows(t, name, x) for t, name in ((x, "x"), (z, "z"), (residual, "residual"))]
    B, H, T = ((1, 1, 1) + x.shape)[-4:-1]
    return KdaNorm(B, H, T, D, code, wcode, _ACTS.get(act, 0), alpha, eps, *strides), dev


def norm_gate_fwd(x, weight=None, z=None, act: str = "silu", residual=None, alpha: float = 1.0, next_weight=None,
                  eps: float = 1e-6, *, s=None, y=None, stream=None):
    """The norms around a block through kda_norm_fwd, over the last dimension (up to 16384 values): (s, y).

        n = x / rms(x) * weight;  h = n * act(z);  s = residual + alpha * h;  y = s / rms(s) * next_weight

    weight None leaves x as it is, z None leaves out the gate, residual None the sum, next_weight None the
    second norm (y is None then).  x, z, residual: up to four dimensions, any strides with a contiguous
    last dimension, bf16 or fp32; weights [D], both bf16 or both fp32; s and y apart from every input (the
    residual is not updated in place).  Asynchronous on `stream`."""
    if stream is not None:
        call = partial(norm_gate_fwd, x, weight, z, act, residual, alpha, next_weight, eps, s=s, y=y)
        return _on_stream(stream, call, x, weight, z, residual, next_weight)
    desc, dev = _norm_inputs(x, weight, z, act, residual, alpha, next_weight, eps)
    if s is None:
        s = _like(x)
    if next_weight is None:
        y = None
    elif y is None:
        y = _like(x)
    ss = _rows(s, "s", x)
    sy = _rows(y, "y", x) if y is not None else ss
    stream = torch.cuda.current_stream(dev.index)
    _call("kda_norm_fwd", dev, (_at(x), _at(weight), _at(z), _at(residual), _at(next_weight), ctypes.byref(desc), _at(s), ctypes.byref(ss),
                                _at(y), ctypes.byref(sy), stream.cuda_stream))
    return s, y


def norm_gate_bwd(x, ds, dy=None, weight=None, z=None, act: str = "silu", residual=None, alpha: float = 1.0, next_weight=None,
                  eps: float = 1e-6, *, workspace=None, stream=None):
    """Gradients of norm_gate_fwd through kda_norm_bwd, given ds = dL/ds (None for zero, with next_weight) and
    dy = dL/dy (with next_weight): (dx, dweight, dz, dresidual, dnext_weight), None for what was not given;
    rows' gradients in x's type, weights' in the weights'.  Asynchronous on `stream`."""
    if stream is not None:
        call = partial(norm_gate_bwd, x, ds, dy, weight, z, act, residual, alpha, next_weight, eps, workspace=workspace)
        return _on_stream(stream, call, x, ds, dy, weight, z, residual, next_weight, workspace)
    desc, dev = _norm_inputs(x, weight, z, act, residual, alpha, next_weight, eps)
    if (dy is None) != (next_weight is None):
        raise ValueError("dy is given exactly when next_weight is")
    if ds is None and next_weight is None:
        raise ValueError("ds is None")
    sds, sdy = (None if t is None else _rows(t, name, x) for t, name in ((ds, "ds"), (dy, "dy")))
    dx = _like(x)
    dz = _like(z) if z is not None else None
    dres = _like(residual) if residual is not None else None
    dw = torch.empty_like(weight) if weight is not None else None
    dw2 = torch.empty_like(next_weight) if next_weight is not None else None
    need = _lib.load().kda_norm_bwd_workspace_bytes(ctypes.byref(desc))
    need = 0 if need == ctypes.c_size_t(-1).value else need
    workspace = _workspace(workspace, need, dev)
    stream = torch.cuda.current_stream(dev.index)
    st = [KdaStride(0, 0, 0) if t is None else _row_strides(t) for t in (dx, dz, dres)]
    grads = KdaNormGrads(_at(dx), _at(dz), _at(dres), _at(dw), _at(dw2), *st)
    ref = lambda t: None if t is None else ctypes.byref(t)  # noqa: E731
    _call("kda_norm_bwd", dev, (_at(x), _at(weight), _at(z), _at(residual), _at(next_weight), ctypes.byref(desc), _at(ds), ref(sds), _at(dy),
                                ref(sdy), ctypes.byref(grads), _at(workspace), need, stream.cuda_stream))
    return dx, dw, dz, dres, dw2
