"""Binding of the operators around the recurrence of a language model:
embedding lookup and gradient, token log probabilities and gradient, linear
attention with a decay for each head (include/rnn355.h has their formulas).

As in the rest of the package this is argument marshalling only.  Work and
allocations of a call go to `stream` (default: the current stream of the
operands' device), so a workspace that a call makes for itself belongs to the
stream that uses it.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from . import RNN_BF16, RNN_F32, RNN_OK, RnnError, load as _load

__all__ = ["embed_fwd", "embed_bwd", "token_logprobs", "token_logprobs_bwd", "linattn_fwd",
           "linattn_step", "linattn_bwd", "LinDims", "workspace_size_embed_bwd",
           "workspace_size_logprobs", "workspace_size_linattn", "OP_LIN_FWD", "OP_LIN_BWD"]

OP_LIN_FWD, OP_LIN_BWD = 0, 1
_DT = {torch.bfloat16: RNN_BF16, torch.float32: RNN_F32}
_IT = {torch.int32: 0, torch.int64: 1}


class _Ids(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("type", ctypes.c_int),
                ("stride_t", ctypes.c_int64), ("stride_b", ctypes.c_int64)]


class _Seq(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride_t", ctypes.c_int64),
                ("stride_b", ctypes.c_int64)]


class LinDims(ctypes.Structure):
    """Dimensions of linear attention (rnn_lin_dims)."""
    _fields_ = [(n, ctypes.c_int) for n in ("T", "B", "NH", "NKV", "Dk", "Dv")]


_declared = None


def load():
    """The library, with the signatures of this module's entry points."""
    global _declared
    lib = _load()
    if lib is _declared:
        return lib
    P, I, S, L, F = (ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_int64,
                     ctypes.c_float)
    ids, seq, dims = ctypes.POINTER(_Ids), ctypes.POINTER(_Seq), ctypes.POINTER(LinDims)
    for name, res, args in (
            ("rnn_embed_fwd", I, [I, I, I, I, I, ids, P, L, F, P, P]),
            ("rnn_workspace_size_embed_bwd", S, [I] * 4),
            ("rnn_embed_bwd", I, [I, I, I, I, I, ids, P, F, P, P, S, P]),
            ("rnn_workspace_size_logprobs", S, [I] * 3),
            ("rnn_token_logprobs", I, [I, I, I, P, L, P, I, I, P, P, P, P, P, P, S, P]),
            ("rnn_token_logprobs_bwd", I, [I, I, I, P, L, P, I, P, P, P, P, P, L, P]),
            ("rnn_workspace_size_linattn", S, [I, dims, I]),
            ("rnn_linattn_fwd", I, [dims, I, seq, seq, seq, P, F, P, P, P, P, S, P]),
            ("rnn_linattn_step", I, [dims, I, seq, seq, seq, P, F, P, P, P, P]),
            ("rnn_linattn_bwd", I, [dims, I, seq, seq, seq, P, F, P, seq, P, P, P, P, P, P, S, P])):
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    _declared = lib
    return lib


def _on_stream(fn):
    """Run with `stream`, and the first operand's device, current."""
    name = fn.__code__.co_varnames[0]

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if not args and name not in kw:
            raise TypeError("%s() missing operand %r" % (fn.__name__, name))
        first = args[0] if args else kw[name]
        if not first.is_cuda:
            raise ValueError("operands must be device tensors")
        if stream is not None:
            if stream.device != first.device:
                raise ValueError("stream is on %s, the operands on %s" % (stream.device, first.device))
            with torch.cuda.stream(stream):
                return fn(*args, **kw)
        if first.get_device() != torch.cuda.current_device():
            with torch.cuda.device(first.device):
                return fn(*args, **kw)
        return fn(*args, **kw)
    return call


# The current stream's handle without the Stream object around it: that costs
# 1.9 us of a call's 11, this 0.1.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _current(dev):
    if _raw_stream is not None:
        return _raw_stream(dev.index)
    return torch.cuda.current_stream(dev).cuda_stream


def _dt(t, name):
    c = _DT.get(t.dtype)
    if c is None:
        raise TypeError("%s must be bfloat16 or float32, got %s" % (name, t.dtype))
    return c


def _it(t, name):
    c = _IT.get(t.dtype)
    if c is None:
        raise TypeError("%s must be int32 or int64, got %s" % (name, t.dtype))
    return c


def _dev(t, name, dev):
    if t.device != dev or not t.is_cuda:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, dev))


def _dense(t, name, dtype, shape, dev) -> Optional[int]:
    """Pointer of a contiguous tensor, None for None."""
    if t is None:
        return None
    _dev(t, name, dev)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _new(t, name, dtype, shape, dev):
    """An output: `t` where given (checked), else a new tensor."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _dense(t, name, dtype, torch.Size(shape), dev)
    return t


def _space(ws, need, dev):
    """(tensor to keep, pointer, bytes) of a workspace of `need` bytes."""
    if need == 0:
        return None, None, 0
    if ws is None or ws.numel() * ws.element_size() < need:
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
    elif not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    _dev(ws, "ws", dev)
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def _ok(s, what):
    if s != RNN_OK:
        raise RnnError(s, what)


# -------------------------------------------------------------- embedding
def _ids(ids, dev):
    _dev(ids, "ids", dev)
    kind = _it(ids, "ids")
    st = ids.stride()
    if len(st) == 1:
        return ids.shape[0], 1, _Ids(ids.data_ptr(), kind, st[0], 0)
    if len(st) != 2:
        raise ValueError("ids must be [T, B] or [M], got %s" % (tuple(ids.shape),))
    T, B = ids.shape
    return T, B, _Ids(ids.data_ptr(), kind, st[0], st[1])


@_on_stream
def embed_fwd(ids, table, scale: float = 1.0, *, out=None):
    """x[t,b,:] = scale * table[ids[t,b],:] in the table's type; ids [T,B] (any
    strides) or [M], int32 or int64; an id outside the table gives zeros.
    table [V,D] with contiguous rows."""
    dev = table.device
    st = table.stride()
    if len(st) != 2 or (st[1] != 1 and table.shape[1] > 1):
        raise ValueError("table must be [V, D] with contiguous rows")
    _dev(table, "table", dev)
    dt = _dt(table, "table")
    T, B, view = _ids(ids, dev)
    V, D = table.shape
    if out is None:
        out = table.new_empty((*ids.shape, D))
    else:
        _new(out, "out", table.dtype, (*ids.shape, D), dev)
    ld = st[0] if V > 1 else D
    _ok(load().rnn_embed_fwd(T, B, V, D, dt, view, table.data_ptr(), ld, scale, out.data_ptr(),
                             _current(dev)), "rnn_embed_fwd")
    return out


def workspace_size_embed_bwd(T: int, B: int, V: int, D: int) -> int:
    return int(load().rnn_workspace_size_embed_bwd(T, B, V, D))


@_on_stream
def embed_bwd(ids, dx, V: int, scale: float = 1.0, *, ws=None, out=None):
    """Gradient of embed_fwd's table: float32 [V,D], every row written; dx
    [*ids.shape, D] bfloat16 or float32."""
    dev = dx.device
    dt = _dt(dx, "dx")
    T, B, view = _ids(ids, dev)
    if dx.dim() != ids.dim() + 1:
        raise ValueError("dx must be [*ids.shape, D]")
    D = dx.shape[-1]
    p = _dense(dx, "dx", dx.dtype, torch.Size((*ids.shape, D)), dev)
    out = _new(out, "out", torch.float32, (V, D), dev)
    ws, wp, wn = _space(ws, workspace_size_embed_bwd(T, B, V, D), dev)
    _ok(load().rnn_embed_bwd(T, B, V, D, dt, view, p, scale, out.data_ptr(), wp, wn,
                             _current(dev)), "rnn_embed_bwd")
    return out


# ------------------------------------------------- token log probabilities
def _rows(t, name):
    """[..., V] as [M, V] rows of contiguous values: (view, row stride)."""
    if t.dim() < 1 or t.shape[-1] == 0:
        raise ValueError("%s must be [..., V]" % name)
    V = t.shape[-1]
    if V > 1 and t.stride(-1) != 1:
        raise ValueError("%s needs contiguous rows" % name)
    r = t if t.dim() == 2 else t.view(-1, V)
    return r, r.stride(0) if r.shape[0] > 1 else V


def workspace_size_logprobs(M: int, V: int, K: int) -> int:
    return int(load().rnn_workspace_size_logprobs(M, V, K))


@_on_stream
def token_logprobs(logits, tokens, top: int = 0, *, ws=None, out=None):
    """Log probability of each row's token, entropy, log-sum-exp and the `top`
    largest entries.  logits [..., V] (rows contiguous, any row stride), tokens
    [...] int32 or int64.  Returns a dict of float32 logp, entropy, lse [...]
    and, with top > 0, top_logp float32 and top_id int32 [..., top]."""
    dev = logits.device
    _dev(logits, "logits", dev)
    dt = _dt(logits, "logits")
    rows, ld = _rows(logits, "logits")
    M, V = rows.shape
    lead = logits.shape[:-1]
    tp = _dense(tokens, "tokens", tokens.dtype, lead, dev)
    names = ("logp", "entropy", "lse")
    if out:
        r = {k: _new(out.get(k), k, torch.float32, lead, dev) for k in names}
    else:  # one allocation for the three
        out = {}
        r = dict(zip(names, torch.empty((3, *lead), dtype=torch.float32, device=dev).unbind()))
    kp = ki = None
    if top:
        r["top_logp"] = _new(out.get("top_logp"), "top_logp", torch.float32, (*lead, top), dev)
        r["top_id"] = _new(out.get("top_id"), "top_id", torch.int32, (*lead, top), dev)
        kp, ki = r["top_logp"].data_ptr(), r["top_id"].data_ptr()
    ws, wp, wn = _space(ws, workspace_size_logprobs(M, V, top), dev)
    _ok(load().rnn_token_logprobs(M, V, dt, rows.data_ptr(), ld, tp, _it(tokens, "tokens"), top,
                                  r["logp"].data_ptr(), r["entropy"].data_ptr(),
                                  r["lse"].data_ptr(), kp, ki, wp, wn, _current(dev)),
        "rnn_token_logprobs")
    return r


@_on_stream
def token_logprobs_bwd(logits, tokens, lse, entropy=None, dlogp=None, dentropy=None, *, out=None):
    """Gradient with respect to the logits, in their type, of
    sum(dlogp * logp) + sum(dentropy * entropy); `out` may be the logits."""
    dev = logits.device
    _dev(logits, "logits", dev)
    dt = _dt(logits, "logits")
    rows, ld = _rows(logits, "logits")
    M, V = rows.shape
    lead = logits.shape[:-1]
    if lse is None:
        raise ValueError("lse is required")
    if dentropy is not None and entropy is None:
        raise ValueError("entropy is required with dentropy")
    tp = _dense(tokens, "tokens", tokens.dtype, lead, dev)
    ps = [_dense(t, n, torch.float32, lead, dev)
          for t, n in ((lse, "lse"), (entropy, "entropy"), (dlogp, "dlogp"), (dentropy, "dentropy"))]
    if out is None:
        out = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
    _dev(out, "out", dev)
    if out.dtype != logits.dtype or out.shape != logits.shape:
        raise ValueError("out must match the logits")
    orows, ldd = _rows(out, "out")
    _ok(load().rnn_token_logprobs_bwd(M, V, dt, rows.data_ptr(), ld, tp, _it(tokens, "tokens"),
                                      *ps, orows.data_ptr(), ldd, _current(dev)),
        "rnn_token_logprobs_bwd")
    return out


# -------------------------------------------------------- linear attention
def _seq(t, name, dtype, dev):
    """[T,B,heads,D] with contiguous [heads,D] rows."""
    _dev(t, name, dev)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.dim() != 4:
        raise ValueError("%s must be [T, B, heads, D]" % name)
    _, _, h, D = t.shape
    st, sb, sh, sd = t.stride()
    if (D > 1 and sd != 1) or (h > 1 and sh != D):
        raise ValueError("%s needs contiguous [heads, D] rows" % name)
    return _Seq(t.data_ptr(), st, sb)


def _lin(q, k, v, g):
    dev = q.device
    dt = _dt(q, "q")
    sq, sk, sv = _seq(q, "q", q.dtype, dev), _seq(k, "k", q.dtype, dev), _seq(v, "v", q.dtype, dev)
    T, B, NH, Dk = q.shape
    NKV, Dv = v.shape[2], v.shape[3]
    if k.shape != (T, B, NKV, Dk) or v.shape[:2] != (T, B):
        raise ValueError("q %s, k %s and v %s do not go together"
                         % (tuple(q.shape), tuple(k.shape), tuple(v.shape)))
    gp = _dense(g, "g", torch.float32, torch.Size((NH,)), dev)
    return LinDims(T, B, NH, NKV, Dk, Dv), dt, sq, sk, sv, gp, dev


def workspace_size_linattn(op: int, dims: LinDims, dtype_code: int) -> int:
    return int(load().rnn_workspace_size_linattn(op, dims, dtype_code))


@_on_stream
def linattn_fwd(q, k, v, g, S0=None, *, scale: Optional[float] = None, ws=None, out=None):
    """Linear attention with a decay for each head over T tokens.  q [T,B,NH,Dk],
    k [T,B,NKV,Dk], v [T,B,NKV,Dv] (views with contiguous [heads, D] rows),
    g [NH] float32 log decays, S0 [B,NH,Dk,Dv] float32 or None (zeros); scale
    defaults to Dk ** -0.5.  Returns (o [T,B,NH,Dv] in q's type, S_T); `out` is
    a dict with "o" and "S" (S may be S0)."""
    d, dt, sq, sk, sv, gp, dev = _lin(q, k, v, g)
    state = torch.Size((d.B, d.NH, d.Dk, d.Dv))
    out = out or {}
    p0 = _dense(S0, "S0", torch.float32, state, dev)
    o = _new(out.get("o"), "o", q.dtype, (d.T, d.B, d.NH, d.Dv), dev)
    S = _new(out.get("S"), "S", torch.float32, state, dev)
    ws, wp, wn = _space(ws, workspace_size_linattn(OP_LIN_FWD, d, dt), dev)
    _ok(load().rnn_linattn_fwd(d, dt, sq, sk, sv, gp, d.Dk ** -0.5 if scale is None else scale, p0,
                               o.data_ptr(), S.data_ptr(), wp, wn, _current(dev)),
        "rnn_linattn_fwd")
    return o, S


@_on_stream
def linattn_step(q, k, v, g, S, *, scale: Optional[float] = None, S_out=None, out=None):
    """One token (T = 1) for each batch row.  The state is updated in place
    unless `S_out` is given.  Returns (o [1,B,NH,Dv], the new state)."""
    d, dt, sq, sk, sv, gp, dev = _lin(q, k, v, g)
    if d.T != 1:
        raise ValueError("linattn_step takes one token, got T = %d" % d.T)
    if S is None:
        raise ValueError("S is required")
    state = torch.Size((d.B, d.NH, d.Dk, d.Dv))
    S_out = S if S_out is None else S_out
    p0 = _dense(S, "S", torch.float32, state, dev)
    p1 = _dense(S_out, "S_out", torch.float32, state, dev)
    o = _new(out, "out", q.dtype, (1, d.B, d.NH, d.Dv), dev)
    _ok(load().rnn_linattn_step(d, dt, sq, sk, sv, gp, d.Dk ** -0.5 if scale is None else scale,
                                p0, o.data_ptr(), p1, _current(dev)), "rnn_linattn_step")
    return o, S_out


@_on_stream
def linattn_bwd(q, k, v, g, do, S0=None, dST=None, *, scale: Optional[float] = None, ws=None,
                out=None):
    """Gradients of sum(do * o) + sum(dST * S_T): dict dq, dk, dv (in q's type,
    dense; shared heads summed) and dS0 float32."""
    d, dt, sq, sk, sv, gp, dev = _lin(q, k, v, g)
    if do.shape != (d.T, d.B, d.NH, d.Dv):
        raise ValueError("do has shape %s, expected %s"
                         % (tuple(do.shape), (d.T, d.B, d.NH, d.Dv)))
    sdo = _seq(do, "do", q.dtype, dev)
    state = torch.Size((d.B, d.NH, d.Dk, d.Dv))
    p0 = _dense(S0, "S0", torch.float32, state, dev)
    pT = _dense(dST, "dST", torch.float32, state, dev)
    out = out or {}
    r = {"dq": _new(out.get("dq"), "dq", q.dtype, q.shape, dev),
         "dk": _new(out.get("dk"), "dk", q.dtype, k.shape, dev),
         "dv": _new(out.get("dv"), "dv", q.dtype, v.shape, dev),
         "dS0": _new(out.get("dS0"), "dS0", torch.float32, state, dev)}
    need = workspace_size_linattn(OP_LIN_BWD, d, dt)
    ws, wp, wn = _space(ws, need, dev)
    _ok(load().rnn_linattn_bwd(d, dt, sq, sk, sv, gp, d.Dk ** -0.5 if scale is None else scale, p0,
                               sdo, pT, *[r[n].data_ptr() for n in ("dq", "dk", "dv", "dS0")], wp,
                               wn, _current(dev)), "rnn_linattn_bwd")
    return r
