"""The operators around the recurrence on the CPU: refusals before anything is
enqueued, workspace sizes, and the tests' own 64-bit definitions against
differences and closed forms."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import gru_recurrence_amd as g  # noqa: E402
from gru_recurrence_amd import lm  # noqa: E402
from tests import lm_ref  # noqa: E402

FAKE = 0x7F0000000000  # never dereferenced: validation fails first
INV, UNS, WSP = g.RNN_ERR_INVALID_ARG, g.RNN_ERR_UNSUPPORTED, 3


def _ids(data=FAKE, kind=1):
    return lm._Ids(data, kind, 4, 1)


def _seq(data=FAKE):
    return lm._Seq(data, 64, 64)


def test_embed_refusals():
    lib = lm.load()
    ok = dict(T=2, B=4, V=10, D=8, dt=1, ids=_ids(), table=FAKE, ld=8, scale=1.0, x=FAKE)

    def fwd(**kw):
        return lib.rnn_embed_fwd(*{**ok, **kw}.values(), None)
    for kw in (dict(T=0), dict(B=0), dict(V=0), dict(D=0), dict(D=-1), dict(dt=2), dict(ids=None),
               dict(ids=_ids(None)), dict(ids=_ids(FAKE + 4)), dict(ids=_ids(FAKE, 2)),
               dict(table=None), dict(table=FAKE + 1), dict(ld=7), dict(x=None), dict(x=FAKE + 2),
               dict(T=1 << 20, B=1 << 11)):
        assert fwd(**kw) == INV, kw
    need = g.workspace_size_embed_bwd(2, 4, 10, 8)
    assert need > 0 and g.workspace_size_embed_bwd(0, 4, 10, 8) == 0
    ok = dict(T=2, B=4, V=10, D=8, dt=0, ids=_ids(), dx=FAKE, scale=1.0, out=FAKE, ws=FAKE, n=need)

    def bwd(**kw):
        return lib.rnn_embed_bwd(*{**ok, **kw}.values(), None)
    for kw in (dict(T=0), dict(dt=5), dict(ids=None), dict(dx=None), dict(dx=FAKE + 4),
               dict(out=None), dict(out=FAKE + 4), dict(ws=FAKE + 8)):
        assert bwd(**kw) == INV, kw
    assert bwd(ws=None) == WSP and bwd(n=need - 1) == WSP


def test_logprobs_refusals():
    lib = lm.load()
    ok = dict(M=4, V=20000, dt=0, x=FAKE, ld=20000, tok=FAKE, it=1, K=5, logp=FAKE, ent=FAKE,
              lse=FAKE, tl=FAKE, ti=FAKE, ws=FAKE, n=1 << 30)

    def fwd(**kw):
        return lib.rnn_token_logprobs(*{**ok, **kw}.values(), None)
    for kw in (dict(M=0), dict(V=0), dict(dt=3), dict(x=None), dict(x=FAKE + 2), dict(ld=19999),
               dict(tok=None), dict(tok=FAKE + 4), dict(it=2), dict(K=-1), dict(K=20001),
               dict(logp=None), dict(tl=None), dict(ti=None), dict(lse=FAKE + 2),
               dict(ent=FAKE + 1), dict(ws=FAKE + 4)):
        assert fwd(**kw) == INV, kw
    assert fwd(K=65) == UNS and fwd(V=1000001, ld=1000001) == UNS
    assert fwd(M=1 << 30, V=999999, ld=1000000) == UNS  # more workgroups than a grid has
    need = g.workspace_size_logprobs(4, 20000, 5)
    assert need > 0 and fwd(n=need - 1) == WSP and fwd(ws=None) == WSP
    assert g.workspace_size_logprobs(4, 100, 5) == 0 and g.workspace_size_logprobs(4, 100, 65) == 0
    ok = dict(M=4, V=100, dt=1, x=FAKE, ld=100, tok=FAKE, it=0, lse=FAKE, ent=FAKE, dl=FAKE,
              de=FAKE, out=FAKE, ldd=100)

    def bwd(**kw):
        return lib.rnn_token_logprobs_bwd(*{**ok, **kw}.values(), None)
    for kw in (dict(M=0), dict(V=0), dict(dt=3), dict(x=None), dict(x=FAKE + 1), dict(ld=99),
               dict(tok=None), dict(tok=FAKE + 2), dict(it=9), dict(lse=None), dict(ent=None),
               dict(lse=FAKE + 2), dict(dl=FAKE + 1), dict(out=None), dict(ldd=99)):
        assert bwd(**kw) == INV, kw
    assert bwd(V=1000001, ld=1000001, ldd=1000001) == UNS


def test_linattn_refusals():
    lib = lm.load()
    D = lm.LinDims
    ok = dict(d=D(500, 1, 4, 2, 64, 64), dt=1, q=_seq(), k=_seq(), v=_seq(), g=FAKE, scale=1.0,
              S0=None, o=FAKE, ST=None, ws=FAKE, n=1 << 40)

    def fwd(**kw):
        return lib.rnn_linattn_fwd(*{**ok, **kw}.values(), None)
    bad_dims = [D(0, 1, 4, 2, 64, 64), D(5, 0, 4, 2, 64, 64), D(5, 1, 0, 1, 64, 64),
                D(5, 1, 4, 0, 64, 64), D(5, 1, 4, 3, 64, 64), D(5, 1, 2, 4, 64, 64),
                D(5, 1, 4, 2, 0, 64), D(5, 1, 4, 2, 64, 0)]
    for d in bad_dims:
        assert fwd(d=d) == INV
    for kw in (dict(dt=2), dict(q=None), dict(k=None), dict(v=None), dict(q=_seq(None)),
               dict(k=_seq(FAKE + 1)), dict(g=None), dict(g=FAKE + 4), dict(o=None),
               dict(o=FAKE + 2), dict(S0=FAKE + 4), dict(ST=FAKE + 8), dict(ws=FAKE + 8)):
        assert fwd(**kw) == INV, kw
    assert fwd(d=D(5, 1, 4, 2, 257, 64)) == UNS and fwd(d=D(5, 1, 4, 2, 64, 257)) == UNS
    need = g.workspace_size_linattn(g.OP_LIN_FWD, ok["d"], 1)
    assert need > 0 and fwd(n=need - 1) == WSP and fwd(ws=None) == WSP
    assert g.workspace_size_linattn(7, ok["d"], 1) == 0
    assert g.workspace_size_linattn(g.OP_LIN_FWD, bad_dims[0], 1) == 0

    sk = dict(d=D(1, 1, 4, 2, 64, 64), dt=1, q=_seq(), k=_seq(), v=_seq(), g=FAKE, scale=1.0,
              S=FAKE, o=FAKE, S1=FAKE)

    def step(**kw):
        return lib.rnn_linattn_step(*{**sk, **kw}.values(), None)
    for kw in (dict(d=D(2, 1, 4, 2, 64, 64)), dict(S=None), dict(S1=None), dict(S=FAKE + 4),
               dict(o=None), dict(q=None), dict(g=None), dict(dt=9)):
        assert step(**kw) == INV, kw
    assert step(d=D(1, 1, 4, 2, 300, 64)) == UNS

    bk = dict(d=D(500, 1, 4, 2, 64, 64), dt=1, q=_seq(), k=_seq(), v=_seq(), g=FAKE, scale=1.0,
              S0=None, do=_seq(), dST=None, dq=FAKE, dk=FAKE, dv=FAKE, dS0=None, ws=FAKE, n=1 << 40)

    def bwd(**kw):
        return lib.rnn_linattn_bwd(*{**bk, **kw}.values(), None)
    for kw in (dict(d=bad_dims[4]), dict(do=None), dict(do=_seq(FAKE + 1)), dict(dq=None),
               dict(dk=None), dict(dv=None), dict(dq=FAKE + 2), dict(dS0=FAKE + 4),
               dict(dST=FAKE + 4)):
        assert bwd(**kw) == INV, kw
    assert bwd(d=D(5, 1, 4, 2, 257, 64)) == UNS
    need = g.workspace_size_linattn(g.OP_LIN_BWD, bk["d"], 1)
    assert need > 0 and bwd(n=need - 1) == WSP


def test_workspace_sizes_do_not_grow_past_the_problem():
    # the carries of embed_bwd: one row per 32 items of M + V
    w = g.workspace_size_embed_bwd(1024, 16, 32000, 768)
    assert w <= 4 * 768 * ((16384 + 32001) // 32 + 2) + 16 * 16384 + (1 << 20)
    # without segments and without shared heads linear attention needs none
    assert g.workspace_size_linattn(g.OP_LIN_FWD, lm.LinDims(64, 1, 1, 1, 64, 64), 1) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    ids, table = torch.zeros((2, 3), dtype=torch.int64), torch.zeros((5, 8))
    with pytest.raises(ValueError):
        g.embed_fwd(ids, table)
    with pytest.raises(ValueError):
        g.token_logprobs(torch.zeros((2, 8)), torch.zeros(2, dtype=torch.int64))
    q = torch.zeros((2, 1, 1, 8))
    with pytest.raises(ValueError):
        g.linattn_fwd(q, q, q, torch.zeros(1))
    with pytest.raises((TypeError, ValueError)):
        g.linattn_fwd(q.double(), q, q, torch.zeros(1))


# ---------------------------------------------- the definitions themselves
def _differences(f, x, rng, h=1e-6):
    v = rng.standard_normal(x.shape)
    return v, (f(x + h * v) - f(x - h * v)) / (2 * h)


def test_reference_gradients_against_differences():
    rng = np.random.default_rng(0)
    T, B, NH, NKV, Dk, Dv = 6, 2, 4, 2, 3, 5
    q, k = rng.standard_normal((T, B, NH, Dk)), rng.standard_normal((T, B, NKV, Dk))
    v, S0 = rng.standard_normal((T, B, NKV, Dv)), rng.standard_normal((B, NH, Dk, Dv))
    ld = -rng.random(NH)
    do, dST = rng.standard_normal((T, B, NH, Dv)), rng.standard_normal((B, NH, Dk, Dv))
    r = lm_ref.linattn_grad(q, k, v, ld, S0, do, dST, 0.7)

    def loss(q=q, k=k, v=v, S0=S0):
        o, S = lm_ref.linattn(q, k, v, ld, S0, 0.7)
        return (o * do).sum() + (S * dST).sum()
    for name, x in (("q", q), ("k", k), ("v", v), ("S0", S0)):
        d, num = _differences(lambda y: loss(**{name: y}), x, rng)
        assert abs(num - (r["d" + name] * d).sum()) < 1e-6 * max(1, abs(num)), name

    x, tok = rng.standard_normal((3, 11)) * 2, np.array([4, 10, -1])
    dl, de = rng.standard_normal(3), rng.standard_normal(3)

    def lloss(y):
        z = lm_ref.logprobs(y, tok, 1)
        return (z["logp"] * dl).sum() + (z["entropy"] * de).sum()
    d, num = _differences(lloss, x, rng)
    assert abs(num - (lm_ref.logprobs_grad(x, tok, dl, de) * d).sum()) < 1e-6


def test_reference_closed_forms():
    # without decay and with unit keys the state is a running sum of values
    v = np.arange(12.0).reshape(4, 1, 1, 3)
    one = np.ones((4, 1, 1, 1))
    o, S = lm_ref.linattn(one, one, v, np.zeros(1), None, 1.0)
    assert np.allclose(o[:, 0, 0], np.cumsum(v[:, 0, 0], 0)) and np.allclose(S[0, 0, 0], v.sum(0)[0, 0])
    # a decay of zero keeps the last token alone
    o, _ = lm_ref.linattn(one, one, v, np.array([-np.inf]), np.ones((1, 1, 1, 3)), 1.0)
    assert np.allclose(o, v)
    r = lm_ref.logprobs(np.zeros((1, 8)), [3], 2)
    assert np.allclose(r["logp"], -np.log(8)) and np.allclose(r["entropy"], np.log(8))
    assert r["top_id"].tolist() == [[0, 1]]
