"""Binding of the operators around the recurrence of a language model:
embedding lookup and gradient, token log probabilities and gradient, linear
attention with a decay for each head, gated linear recurrence, gradient norm
and clipping, verification of drafted tokens (include/rnn355.h has their
formulas).

As in the rest of the package this is argument marshalling only.  Work and
allocations of a call go to `stream` (default: the current stream of the
operands' device), so a workspace that a call makes for itself belongs to the
stream that uses it.
"""
from __future__ import annotations

import array
import ctypes
import functools
import itertools
import operator
from typing import Optional

import torch

from . import RNN_BF16, RNN_ERR_INVALID_ARG, RNN_F32, RNN_OK, RnnError, load as _load

__all__ = ["embed_fwd", "embed_bwd", "token_logprobs", "token_logprobs_bwd", "linattn_fwd",
           "linattn_step", "linattn_bwd", "LinDims", "workspace_size_embed_bwd",
           "workspace_size_logprobs", "workspace_size_linattn", "OP_LIN_FWD", "OP_LIN_BWD",
           "gated_fwd", "gated_step", "gated_bwd", "GatedDims", "workspace_size_gated",
           "OP_GATED_FWD", "OP_GATED_BWD", "grad_norm", "clip_grads", "GradList",
           "workspace_size_clip", "verify_drafts", "workspace_size_verify"]

OP_LIN_FWD, OP_LIN_BWD = 0, 1
OP_GATED_FWD, OP_GATED_BWD = 0, 1
_GATES = {"logit": 0, "decay": 1}
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


class GatedDims(ctypes.Structure):
    """Dimensions of the gated linear recurrence (rnn_gated_dims)."""
    _fields_ = [(n, ctypes.c_int) for n in ("T", "B", "D")]


class _Grad(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("out", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("dtype", ctypes.c_int)]


_declared = None


def load():
    """The library, with the signatures of this module's entry points."""
    global _declared
    lib = _load()
    if lib is _declared:
        return lib
    P, I, S, L, F, D = (ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_int64,
                        ctypes.c_float, ctypes.c_double)
    ids, seq, dims = ctypes.POINTER(_Ids), ctypes.POINTER(_Seq), ctypes.POINTER(LinDims)
    gated, grads = ctypes.POINTER(GatedDims), P  # rnn_grad[count] as its bytes
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
            ("rnn_linattn_bwd", I, [dims, I, seq, seq, seq, P, F, P, seq, P, P, P, P, P, P, S, P]),
            ("rnn_workspace_size_gated", S, [I, gated, I]),
            ("rnn_gated_fwd", I, [gated, I, I, seq, seq, P, P, seq, P, P, S, P]),
            ("rnn_gated_step", I, [gated, I, I, seq, seq, P, seq, P, P]),
            ("rnn_gated_bwd", I, [gated, I, I, seq, seq, seq, seq, P, P, P, seq, seq, P, P, S, P]),
            ("rnn_workspace_size_clip", S, [I, grads]),
            ("rnn_grad_norm", I, [I, grads, P, P, S, P]),
            ("rnn_clip_grads", I, [I, grads, D, P, P, S, P]),
            ("rnn_workspace_size_verify", S, [I] * 3),
            ("rnn_verify_drafts", I, [I, I, I, I, seq, ids, seq, P, P, P, P, P, P, S, P])):
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    _declared = lib
    return lib


# The current device's number; the plain call checks each time that CUDA is
# initialised, which an operand on it says already.
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


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
        if first.get_device() != _device():
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


# ------------------------------------------------- gated linear recurrence
def _row(t, name, dtype, shape, dev):
    """[T,B,D] with contiguous rows, any other strides."""
    if t.device != dev:
        _dev(t, name, dev)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    st, sb, sd = t.stride()
    if sd != 1 and shape[2] > 1:
        raise ValueError("%s needs contiguous rows of D values" % name)
    return _Seq(t.data_ptr(), st, sb)


def _row_out(t, name, dtype, shape, dev, like=None):
    """An output sequence: (tensor, view); a view given must not overlap itself.
    `like`: an operand of its type and shape, for a new one."""
    if t is None:
        t = torch.empty_like(like, memory_format=torch.contiguous_format)  # 0.9 us less than empty(shape)
        return t, _Seq(t.data_ptr(), shape[1] * shape[2], shape[2])
    v = _row(t, name, dtype, shape, dev)
    need = shape[2]
    for step, n in sorted(((v.stride_t, shape[0]), (v.stride_b, shape[1]))):
        if n > 1:
            if step < need:
                raise ValueError("rows of %s overlap" % name)
            need += step * (n - 1)
    return t, v


def _state(t, name, shape, dev):
    """Pointer of a contiguous float32 state, None for None."""
    if t is None:
        return None
    if t.dtype != torch.float32 or t.shape != shape or t.device != dev or not t.is_contiguous():
        _dense(t, name, torch.float32, shape, dev)  # says what is wrong
    return t.data_ptr()


def _refused(s, what, **states):
    """Raises what a call of the gated recurrence was refused for."""
    for name, t in states.items():
        if s == RNN_ERR_INVALID_ARG and t is not None and t.data_ptr() % 16:
            raise ValueError("%s must start at a multiple of 16 bytes (a row of a larger tensor may not)" % name)
    raise RnnError(s, what)


def _gated(f, x, gate, lens):
    dev, shape, dtype = f.device, f.shape, f.dtype
    dt, gt = _dt(f, "f"), _GATES.get(gate)
    if gt is None:
        raise ValueError("gate must be 'logit' or 'decay', got %r" % (gate,))
    if len(shape) != 3:
        raise ValueError("f must be [T, B, D], got %s" % (tuple(shape),))
    sf = _row(f, "f", dtype, shape, dev)
    sx = None if x is None else _row(x, "x", dtype, shape, dev)
    T, B, D = shape
    lp = None if lens is None else _dense(lens, "lens", torch.int32, (B,), dev)
    return (T, B, D), dt, gt, sf, sx, lp, shape, dev


@functools.lru_cache(maxsize=256)
def _gated_space(op, T, B, D, dt):
    return workspace_size_gated(op, GatedDims(T, B, D), dt)


def workspace_size_gated(op: int, dims: GatedDims, dtype_code: int) -> int:
    return int(load().rnn_workspace_size_gated(op, dims, dtype_code))


@_on_stream
def gated_fwd(f, x, h0=None, *, gate: str = "logit", lens=None, ws=None, out=None):
    """Gated linear recurrence over T tokens, elementwise in [T,B,D] views with
    contiguous rows: gate "logit" h_t = a h_{t-1} + (1 - a) x_t with a =
    sigmoid(f_t) (-inf begins a sequence), gate "decay" h_t = f_t h_{t-1} + x_t.
    h0 [B,D] float32 or None (zeros; states start at a multiple of 16 bytes); lens
    [B] int32: tokens of each row that count (h is 0 behind them).
    Returns (h [T,B,D] in f's type, h_T [B,D] float32, the state behind the last
    token that counts); `out` is a dict with "h" (any view) and "hT" (may be h0).
    A wait between segments that runs out (seconds) is noted in the workspace:
    workspace_status(ws), for a `ws` of workspace_size_gated bytes given here."""
    if x is None:
        raise ValueError("x is required")
    (T, B, D), dt, gt, sf, sx, lp, shape, dev = _gated(f, x, gate, lens)
    state = (B, D)
    out = out or {}
    p0 = _state(h0, "h0", state, dev)
    h, sh = _row_out(out.get("h"), "h", f.dtype, shape, dev, f)
    hT = _new(out.get("hT"), "hT", torch.float32, state, dev)
    ws, wp, wn = _space(ws, _gated_space(OP_GATED_FWD, T, B, D, dt), dev)
    s = load().rnn_gated_fwd(GatedDims(T, B, D), dt, gt, sf, sx, p0, lp, sh, hT.data_ptr(), wp, wn, _current(dev))
    if s != RNN_OK:
        _refused(s, "rnn_gated_fwd", h0=h0, hT=hT)
    return h, hT


@_on_stream
def gated_step(f, x, h, *, gate: str = "logit", h_out=None, out=None):
    """One token (T = 1) for each batch row.  The state h [B,D] float32 is updated
    in place unless `h_out` is given.  Returns (its rounding [1,B,D] in f's type,
    the new state)."""
    if x is None or h is None:
        raise ValueError("x and h are required")
    (T, B, D), dt, gt, sf, sx, _, shape, dev = _gated(f, x, gate, None)
    if T != 1:
        raise ValueError("gated_step takes one token, got T = %d" % T)
    p0 = _state(h, "h", (B, D), dev)
    if h_out is None:
        h_out, p1 = h, p0
    else:
        p1 = _state(h_out, "h_out", (B, D), dev)
    y, sy = _row_out(out, "out", f.dtype, shape, dev, f)
    s = load().rnn_gated_step(GatedDims(T, B, D), dt, gt, sf, sx, p0, sy, p1, _current(dev))
    if s != RNN_OK:
        _refused(s, "rnn_gated_step", h=h, h_out=h_out)
    return y, h_out


@_on_stream
def gated_bwd(f, x, h, dh, h0=None, dhT=None, *, gate: str = "logit", lens=None, ws=None, out=None):
    """Gradients of sum(dh * h) + sum(dhT * h_T), given gated_fwd's h: dict df, dx
    (in f's type) and dh0 float32.  x may be None with gate "decay"; `out` is a
    dict with "df", "dx" (any views) and "dh0" (may be dhT).  workspace_status(ws)
    as in gated_fwd."""
    (T, B, D), dt, gt, sf, sx, lp, shape, dev = _gated(f, x, gate, lens)
    if x is None and gt == 0:
        raise ValueError("x is required with gate 'logit'")
    sh, sdh = _row(h, "h", f.dtype, shape, dev), _row(dh, "dh", f.dtype, shape, dev)
    state = (B, D)
    p0 = _state(h0, "h0", state, dev)
    pT = _state(dhT, "dhT", state, dev)
    out = out or {}
    df, sdf = _row_out(out.get("df"), "df", f.dtype, shape, dev, f)
    dx, sdx = _row_out(out.get("dx"), "dx", f.dtype, shape, dev, f)
    dh0 = _new(out.get("dh0"), "dh0", torch.float32, state, dev)
    ws, wp, wn = _space(ws, _gated_space(OP_GATED_BWD, T, B, D, dt), dev)
    s = load().rnn_gated_bwd(GatedDims(T, B, D), dt, gt, sf, sx, sh, sdh, p0, pT, lp, sdf, sdx, dh0.data_ptr(), wp,
                             wn, _current(dev))
    if s != RNN_OK:
        _refused(s, "rnn_gated_bwd", h0=h0, dhT=dhT, dh0=dh0)
    return {"df": df, "dx": dx, "dh0": dh0}


# ------------------------------------------------ gradient norm, clipping
_get_dtype, _get_shape = operator.attrgetter("dtype"), operator.attrgetter("shape")


class GradList:
    """Gradients checked once, for programs whose gradient buffers stay where they
    are: `grads` are contiguous bfloat16 or float32 tensors of one device, `out`
    (None: in place) tensors of the same types and shapes.  For clipping an output
    may be its own gradient, but not overlap another one or another output."""

    def __init__(self, grads, out=None):
        grads = list(grads)
        if not grads:
            raise ValueError("an empty list of gradients")
        self.device = dev = grads[0].device
        self.is_cuda = grads[0].is_cuda
        if not self.is_cuda:
            raise ValueError("operands must be device tensors")
        outs = grads if out is None else list(out)
        if len(outs) != len(grads):
            raise ValueError("%d outputs for %d gradients" % (len(outs), len(grads)))
        # a list at a time: half the time of a tensor at a time
        n, at = list(map(torch.Tensor.numel, grads)), list(map(torch.Tensor.data_ptr, grads))
        types = list(map(_get_dtype, grads))
        codes = list(map(_DT.get, types))
        if None in codes:
            raise TypeError("gradients must be bfloat16 or float32, got %s" % types[codes.index(None)])
        if set(map(torch.Tensor.get_device, grads)) != {dev.index} or not all(map(torch.Tensor.is_contiguous, grads)):
            raise ValueError("gradients must be contiguous tensors of one device")
        to = at
        if out is not None:
            if (list(map(_get_dtype, outs)) != types
                    or list(map(_get_shape, outs)) != list(map(_get_shape, grads))
                    or set(map(torch.Tensor.get_device, outs)) != {dev.index}
                    or not all(map(torch.Tensor.is_contiguous, outs))):
                raise ValueError("outputs must match their gradients")
            to = list(map(torch.Tensor.data_ptr, outs))
        written = [p for p, k in zip(to, n) if k]
        self.grads, self.out, self.count = grads, outs, len(grads)
        self.twice = len(set(written)) != len(written)
        # rnn_grad has four fields of 8 bytes (the type's upper half is padding)
        self._rows = array.array("q", itertools.chain.from_iterable(zip(at, to, n, codes)))
        self.array = self._rows.buffer_info()[0]

    def get_device(self):
        return self.device.index


def workspace_size_clip(grads) -> int:
    g = grads if isinstance(grads, GradList) else GradList(grads)
    return int(load().rnn_workspace_size_clip(g.count, g.array))


@_on_stream
def _clip(g, max_norm, norm, ws):
    dev, lib = g.device, load()
    norm = _new(norm, "norm", torch.float32, (), dev)
    ws, wp, wn = _space(ws, int(lib.rnn_workspace_size_clip(g.count, g.array)), dev)
    if max_norm is None:
        _ok(lib.rnn_grad_norm(g.count, g.array, norm.data_ptr(), wp, wn, _current(dev)),
            "rnn_grad_norm")
    else:
        s = lib.rnn_clip_grads(g.count, g.array, max_norm, norm.data_ptr(), wp, wn, _current(dev))
        if s == RNN_ERR_INVALID_ARG and wp % 16 == 0:  # all else is checked
            raise ValueError("an output, or norm, overlaps another tensor")
        _ok(s, "rnn_clip_grads")
    return norm


def grad_norm(grads, *, norm=None, ws=None, stream=None):
    """Global 2-norm of a list of gradients (or a GradList): a float32 scalar on
    their device, written to `norm` where given."""
    g = grads if isinstance(grads, GradList) else GradList(grads)
    return _clip(g, None, norm, ws, stream=stream)


def clip_grads(grads, max_norm: float, *, out=None, norm=None, ws=None, stream=None):
    """Scale gradients by max_norm / norm where their global 2-norm exceeds
    max_norm, in place or into the tensors of `out` (a GradList brings its own),
    none of which may overlap another gradient or output.  Returns the norm before that, a float32 scalar on the device; where it is not
    finite the gradients stay as they are."""
    if isinstance(grads, GradList):
        if out is not None:
            raise ValueError("a GradList brings its own outputs")
        g = grads
    else:
        g = GradList(grads, out)
    if g.twice:
        raise ValueError("the same output more than once")
    if not max_norm >= 0:
        raise ValueError("max_norm must be 0 or more, got %r" % (max_norm,))
    return _clip(g, float(max_norm), norm, ws, stream=stream)


# ------------------------------------------- verification of drafted tokens
def workspace_size_verify(K: int, B: int, V: int) -> int:
    return int(load().rnn_workspace_size_verify(K, B, V))


_verify_space = functools.lru_cache(maxsize=256)(workspace_size_verify)


@_on_stream
def verify_drafts(logits, drafts, u, draft_logits=None, *, temperature=None, n_drafts=None, ws=None,
                  out=None):
    """Verify drafted tokens against the target's logits, so that what comes out is
    distributed as the target's own.  logits [K+1,B,V] (rows contiguous), drafts
    [K,B] int32 or int64 (any strides), u [K+1,B] float32 uniform numbers: u[k]
    tests draft k, u[K] draws the token behind the accepted ones.  draft_logits
    [K,B,V] the logits the drafts were drawn from (None: found some other way);
    temperature [B] float32 (0 or less: greedy), n_drafts [B] int32 (None: K).
    Returns (tokens [K+1,B] int32: accepted drafts, the drawn token, then -1;
    accepted [B] int32); `out` is a dict with "tokens" and "accepted".  A wait
    that runs out draws -1; workspace_status(ws) says so, for a `ws` of
    workspace_size_verify bytes given here."""
    dev, shape = logits.device, logits.shape
    dt = _dt(logits, "logits")
    if len(shape) != 3 or 0 in shape:
        raise ValueError("logits must be [K+1, B, V], got %s" % (tuple(shape),))
    R, B, V = shape
    K = R - 1
    sl = _row(logits, "logits", logits.dtype, shape, dev)
    view = sq = None
    if K:
        if drafts is None or drafts.shape != (K, B):
            raise ValueError("drafts must be [K, B] = [%d, %d]" % (K, B))
        view = _ids(drafts, dev)[2]
        if draft_logits is not None:
            sq = _row(draft_logits, "draft_logits", logits.dtype, (K, B, V), dev)
    if u is None:
        raise ValueError("u is required")
    up = _state(u, "u", (R, B), dev)
    tp = _state(temperature, "temperature", (B,), dev)
    np_ = _dense(n_drafts, "n_drafts", torch.int32, (B,), dev)
    out = out or {}
    tokens = _new(out.get("tokens"), "tokens", torch.int32, (R, B), dev)
    accepted = _new(out.get("accepted"), "accepted", torch.int32, (B,), dev)
    ws, wp, wn = _space(ws, _verify_space(K, B, V), dev)
    _ok(load().rnn_verify_drafts(K, B, V, dt, sl, view, sq, up, tp, np_, tokens.data_ptr(),
                                 accepted.data_ptr(), wp, wn, _current(dev)), "rnn_verify_drafts")
    return tokens, accepted
