"""Gated linear recurrence, gradient clipping and draft verification on the CPU:
refusals before anything is enqueued, workspace sizes, how the binding takes its
arguments, and the tests' own 64-bit definitions."""
import inspect

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import gru_recurrence_amd as g  # noqa: E402
from gru_recurrence_amd import lm  # noqa: E402
from tests import gated_ref  # noqa: E402

FAKE = 0x7F0000000000  # never dereferenced: validation fails first
INV, UNS, WSP = g.RNN_ERR_INVALID_ARG, g.RNN_ERR_UNSUPPORTED, 3
BIG = 1 << 60


def _seq(data=FAKE, st=64, sb=64):
    return lm._Seq(data, st, sb)


def test_gated_refusals():
    lib, D = lm.load(), lm.GatedDims
    ok = dict(d=D(100, 2, 64), dt=1, gate=0, f=_seq(), x=_seq(), h0=None, lens=None, h=_seq(), hT=None,
              ws=FAKE, n=BIG)

    def fwd(**kw):
        return lib.rnn_gated_fwd(*{**ok, **kw}.values(), None)
    bad_dims = [D(0, 1, 4), D(1, 0, 4), D(1, 1, 0), D(-1, 1, 1), D(1 << 20, 1 << 11, 1)]
    for d in bad_dims:
        assert fwd(d=d) == INV
        assert g.workspace_size_gated(g.OP_GATED_FWD, d, 0) == 0
    for kw in (dict(d=None), dict(dt=2), dict(gate=2), dict(f=None), dict(x=None), dict(h=None),
               dict(f=_seq(None)), dict(x=_seq(FAKE + 1)), dict(h=_seq(FAKE + 1)), dict(h0=FAKE + 4),
               dict(hT=FAKE + 8), dict(lens=FAKE + 2), dict(ws=FAKE + 4)):
        assert fwd(**kw) == INV, kw
    wide = D(1, 1 << 11, 1 << 20)
    assert fwd(d=wide) == UNS and g.workspace_size_gated(g.OP_GATED_FWD, wide, 1) == 0
    assert g.workspace_size_gated(7, ok["d"], 1) == 0 and g.workspace_size_gated(0, ok["d"], 5) == 0

    sk = dict(d=D(1, 2, 64), dt=0, gate=1, f=_seq(), x=_seq(), h=FAKE, y=_seq(), h_out=FAKE)

    def step(**kw):
        return lib.rnn_gated_step(*{**sk, **kw}.values(), None)
    for kw in (dict(d=D(2, 2, 64)), dict(dt=3), dict(gate=-1), dict(f=None), dict(x=None), dict(h=None),
               dict(h_out=None), dict(h=FAKE + 4), dict(h_out=FAKE + 4), dict(y=_seq(FAKE + 2))):
        assert step(**kw) == INV, kw
    assert step(d=wide) == UNS

    bk = dict(d=D(100, 2, 64), dt=1, gate=0, f=_seq(), x=_seq(), h=_seq(), dh=_seq(), h0=None, dhT=None,
              lens=None, df=_seq(), dx=_seq(), dh0=None, ws=FAKE, n=BIG)

    def bwd(**kw):
        return lib.rnn_gated_bwd(*{**bk, **kw}.values(), None)
    for kw in (dict(d=bad_dims[2]), dict(dt=9), dict(gate=5), dict(f=None), dict(x=None), dict(h=None),
               dict(dh=None), dict(df=None), dict(dx=None), dict(dh=_seq(FAKE + 1)),
               dict(df=_seq(None)), dict(dhT=FAKE + 4), dict(dh0=FAKE + 4), dict(lens=FAKE + 1),
               dict(gate=1, x=_seq(FAKE + 1))):
        assert bwd(**kw) == INV, kw
    assert bwd(d=wide) == UNS


@pytest.mark.parametrize("op", [g.OP_GATED_FWD, g.OP_GATED_BWD])
def test_gated_workspace_is_asked_for(op):
    lib, d = lm.load(), lm.GatedDims(5000, 1, 64)
    need = g.workspace_size_gated(op, d, 1)
    if need == 0:
        return
    s = [_seq()] * 2
    for ws, n in ((None, BIG), (FAKE, need - 1)):
        if op == g.OP_GATED_FWD:
            r = lib.rnn_gated_fwd(d, 1, 0, *s, None, None, _seq(), None, ws, n, None)
        else:
            r = lib.rnn_gated_bwd(d, 1, 0, *s, *s, None, None, None, *s, None, ws, n, None)
        assert r == WSP
    # a single token needs none
    assert g.workspace_size_gated(op, lm.GatedDims(1, 8, 64), 1) == 0


@pytest.mark.parametrize("dt", [g.RNN_F32, g.RNN_BF16])
@pytest.mark.parametrize("T,B,D", [(1024, 1 << 20, 1024), (1 << 15, 1 << 15, 1 << 15), (1 << 10, 1 << 20, 600)])
def test_gated_launches_past_2_32_threads(T, B, D, dt):
    lib, d, s = lm.load(), lm.GatedDims(T, B, D), [_seq()] * 2
    assert T * B <= 1 << 30 and B * D <= 1 << 30
    assert lib.rnn_gated_fwd(d, dt, 0, *s, None, None, _seq(), None, FAKE, BIG, None) == UNS
    assert lib.rnn_gated_bwd(d, dt, 0, *s, *s, None, None, None, *s, None, FAKE, BIG, None) == UNS
    assert g.workspace_size_gated(g.OP_GATED_FWD, d, dt) == 0


def _list(*rows):
    return (lm._Grad * len(rows))(*rows)


def test_clip_refusals():
    lib = lm.load()
    good = _list((FAKE, FAKE, 100, 0), (FAKE, None, 7, 1), (None, None, 0, 1))
    need = lib.rnn_workspace_size_clip(3, good)
    assert need > 0

    def clip(count=3, lst=good, max_norm=1.0, norm=FAKE, ws=FAKE, n=need):
        return lib.rnn_clip_grads(count, lst, max_norm, norm, ws, n, None)

    def norm(count=3, lst=good, norm=FAKE, ws=FAKE, n=need):
        return lib.rnn_grad_norm(count, lst, norm, ws, n, None)
    bad = [_list((None, None, 5, 0)), _list((FAKE + 2, None, 5, 0)), _list((FAKE + 1, None, 5, 1)),
           _list((FAKE, FAKE + 2, 5, 0)), _list((FAKE, None, -1, 0)), _list((FAKE, None, 5, 2)),
           _list((FAKE, None, (1 << 40) + 1, 1))]
    for b in bad:
        assert clip(1, b) == INV and norm(1, b) == INV
        assert lib.rnn_workspace_size_clip(1, b) == 0
    half = (FAKE, None, (1 << 39) + 1, 1)
    assert clip(2, _list(half, half)) == INV
    for f in (clip, norm):
        assert f(count=0) == INV and f(lst=None) == INV and f(norm=None) == INV
        assert f(norm=FAKE + 2) == INV and f(ws=FAKE + 8) == INV
        assert f(ws=None) == WSP and f(n=need - 1) == WSP
    for m in (-1.0, float("nan")):
        assert clip(max_norm=m) == INV


def test_verify_refusals():
    lib = lm.load()
    ids = lm._Ids(FAKE, 1, 4, 1)
    need = g.workspace_size_verify(3, 4, 20000)
    ok = dict(K=3, B=4, V=20000, dt=0, l=_seq(), d=ids, q=_seq(), u=FAKE, t=None, n=None, tok=FAKE,
              acc=FAKE, ws=FAKE, bytes=need)

    def call(**kw):
        return lib.rnn_verify_drafts(*{**ok, **kw}.values(), None)
    for kw in (dict(K=-1), dict(B=0), dict(V=0), dict(dt=2), dict(l=None), dict(l=_seq(None)),
               dict(l=_seq(FAKE + 2)), dict(d=None), dict(d=lm._Ids(None, 1, 4, 1)),
               dict(d=lm._Ids(FAKE, 3, 4, 1)), dict(d=lm._Ids(FAKE + 4, 1, 4, 1)),
               dict(q=_seq(FAKE + 1)), dict(q=_seq(None)), dict(u=None), dict(u=FAKE + 2),
               dict(t=FAKE + 1), dict(n=FAKE + 3), dict(tok=None), dict(acc=None), dict(tok=FAKE + 1),
               dict(ws=FAKE + 8), dict(K=62, B=1 << 25)):
        assert call(**kw) == INV, kw
    assert need > 0 and call(ws=None) == WSP and call(bytes=need - 1) == WSP
    assert call(K=64) == UNS and call(V=1000001) == UNS and call(K=7, B=1 << 20, V=20000) == UNS
    assert g.workspace_size_verify(64, 1, 10) == 0 and g.workspace_size_verify(1, 1, 1000001) == 0
    assert g.workspace_size_verify(-1, 1, 10) == 0


# --------------------------------------------------------------- the binding
def _args(op):
    t, s = torch.zeros((1, 2, 8)), torch.zeros((2, 8))
    return {"gated_fwd": dict(f=t, x=t), "gated_step": dict(f=t, x=t, h=s),
            "gated_bwd": dict(f=t, x=t, h=t, dh=t), "grad_norm": dict(grads=[t]),
            "clip_grads": dict(grads=[t], max_norm=1.0),
            "verify_drafts": dict(logits=t, drafts=torch.zeros((0, 2), dtype=torch.int64),
                                  u=torch.zeros((1, 2)))}[op]


OPS = ("gated_fwd", "gated_step", "gated_bwd", "grad_norm", "clip_grads", "verify_drafts")


@pytest.mark.parametrize("op", OPS)
def test_operands_by_name_and_from_the_host(op):
    a = _args(op)
    with pytest.raises(ValueError, match="device tensor"):
        getattr(g, op)(**a)
    with pytest.raises(ValueError, match="device tensor"):
        getattr(g, op)(*a.values())
    names = list(inspect.signature(getattr(g, op)).parameters)
    assert names[:len(a)] == list(a)
    with pytest.raises(TypeError, match=names[0]):
        getattr(g, op)()


@pytest.mark.parametrize("op", OPS[:3] + OPS[5:])
def test_stream_of_another_device(op):
    class Stream:
        device = torch.device("cuda", 1)

    class Operand:
        device, is_cuda = torch.device("cuda", 0), True
    rest = list(_args(op).values())[1:]
    with pytest.raises(ValueError, match="stream"):
        getattr(g, op)(Operand(), *rest, stream=Stream())


def test_empty_list():
    for f in (g.grad_norm, lambda x: g.clip_grads(x, 1.0), g.GradList):
        with pytest.raises(ValueError, match="empty"):
            f([])


def test_output_rows_must_not_overlap():
    dev = torch.device("cpu")
    f32 = torch.float32

    def view(shape, strides):
        return torch.zeros(1000).as_strided(shape, strides)
    for shape, strides in (((4, 3, 5), (15, 5, 1)), ((4, 3, 5), (5, 20, 1)), ((4, 3, 5), (40, 7, 1)),
                           ((1, 3, 5), (0, 5, 1)), ((4, 1, 5), (5, 0, 1)), ((1, 1, 5), (0, 0, 1)),
                           ((4, 3, 1), (3, 1, 1))):
        lm_row = _unchecked_device(lambda: lm._row_out(view(shape, strides), "o", f32, torch.Size(shape), dev))
        assert lm_row[1].stride_t == strides[0] and lm_row[1].stride_b == strides[1]
    for shape, strides in (((4, 3, 5), (15, 4, 1)), ((4, 3, 5), (14, 5, 1)), ((4, 3, 5), (0, 5, 1)),
                           ((4, 3, 5), (5, 5, 1)), ((4, 3, 5), (5, 19, 1)), ((4, 1, 5), (4, 0, 1)),
                           ((4, 3, 5), (15, 5, 2))):
        with pytest.raises(ValueError):
            _unchecked_device(lambda: lm._row_out(view(shape, strides), "o", f32, torch.Size(shape), dev))


def _unchecked_device(f):
    keep, lm._dev = lm._dev, lambda *a: None
    try:
        return f()
    finally:
        lm._dev = keep


# ---------------------------------------------- the definitions themselves
@pytest.mark.parametrize("gate", ["logit", "decay"])
def test_reference_gradient_against_differences(gate):
    rng = np.random.default_rng(0)
    T, B, D = 7, 3, 4
    f, x, dh = (rng.standard_normal((T, B, D)) for _ in range(3))
    h0, dhT = rng.standard_normal((B, D)), rng.standard_normal((B, D))
    lens = [7, 0, 4]

    def loss(f=f, x=x, h0=h0):
        h, S, _, _ = gated_ref.gated(f, x, h0, gate, lens)
        return (h * dh).sum() + (S * dhT).sum()
    h = gated_ref.gated(f, x, h0, gate, lens)[0]
    r, _ = gated_ref.gated_grad(f, x, h, dh, h0, dhT, gate, lens)
    for k, v in (("f", f), ("x", x), ("h0", h0)):
        d, e = rng.standard_normal(v.shape), 1e-6
        num = (loss(**{k: v + e * d}) - loss(**{k: v - e * d})) / (2 * e)
        assert abs(num - (r["d" + k] * d).sum()) < 1e-7 * max(1, abs(num)), k


def test_reference_closed_forms():
    one = np.ones((6, 1, 1))
    h, S, _, _ = gated_ref.gated(one, one, None, "decay")
    assert np.allclose(h[:, 0, 0], np.arange(1, 7)) and np.allclose(S, 6)
    # a gate half open averages with the state
    h, _, _, _ = gated_ref.gated(0 * one, one, np.zeros((1, 1)), "logit")
    assert np.allclose(h[:, 0, 0], 1 - 0.5 ** np.arange(1, 7))
    n, r = gated_ref.clip([np.array([3.0]), np.array([[4.0]])], 1.0)
    assert n == 5 and np.allclose([r[0][0], r[1][0, 0]], [0.6, 0.8])


def test_reference_verification_keeps_the_target_distribution():
    """Summed over all drafts and a fine grid of uniform numbers, the first token
    is distributed as p."""
    p, q = np.array([0.5, 0.2, 0.3]), np.array([0.1, 0.6, 0.3])
    n, got = 400, np.zeros(3)
    grid = (np.arange(n) + 0.5) / n
    lp, lq = np.log(p), np.log(q)
    for x in range(3):
        u = np.stack([np.repeat(grid, 40), np.tile((np.arange(40) + 0.5) / 40, n)])
        B = u.shape[1]
        tok, _ = gated_ref.verify(np.broadcast_to(lp, (2, B, 3)), np.full((1, B), x), u,
                                  np.broadcast_to(lq, (1, B, 3)))
        got += q[x] * np.bincount(tok[0], minlength=3) / B
    # the grids' spacing: half a step of either
    assert np.abs(got - p).max() <= 1.0 / n + 1.0 / 40
