"""Ends of the ranges of the gated recurrence, gradient clipping and draft
verification: what their workspaces report, values near float32's largest, logits
that are infinite, roundings next to a border, equal rows at different places."""
import numpy as np
import pytest

from tests import gated_ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gru_recurrence_amd as g  # noqa: E402
from tests.test_gpu_gated import _np, _within  # noqa: E402

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _odd(t):
    """The same values in rows that start at an odd element."""
    return torch.nn.functional.pad(t, (1, 2 - t.shape[-1] % 2))[..., 1:t.shape[-1] + 1]


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("T,B,D", [(1024, 16, 768), (600, 24, 500), (100, 32, 700), (300, 10, 1024)])
def test_gated_status_is_ok_on_a_workspace_holding_garbage(T, B, D, odd):
    """Whatever plan the operands' alignment gives a call that asks for a workspace,
    it leaves the status word of that call there."""
    gen = torch.Generator(device="cuda").manual_seed(T)
    f, x, dh = (torch.randn((T, B, D), generator=gen, device="cuda").bfloat16() for _ in range(3))
    if odd:
        f, x, dh = _odd(f), _odd(x), _odd(dh)
    d = g.GatedDims(T, B, D)
    need = [g.workspace_size_gated(op, d, g.RNN_BF16) for op in (g.OP_GATED_FWD, g.OP_GATED_BWD)]
    assert max(need) > 0
    h, _ = g.gated_fwd(f, x)
    for n, call in zip(need, (lambda w: g.gated_fwd(f, x, ws=w), lambda w: g.gated_bwd(f, x, h, dh, ws=w))):
        if n == 0:
            continue
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        call(ws)
        assert g.workspace_status(ws) == g.RNN_OK


def _huge(T, B, D, dt, seed):
    """Values up to near the type's largest with both signs, logits of any size and
    infinite ones."""
    rng = np.random.default_rng(seed)
    f = 4.0 * rng.standard_normal((T, B, D))
    pick = rng.random((T, B, D))
    f[pick < 0.15], f[pick > 0.85] = -np.inf, np.inf

    def big(shape):
        return rng.choice([-1.0, 1.0], shape) * 10.0 ** rng.uniform(37.0, 38.5, shape)
    x, h0 = big((T, B, D)), big((B, D))
    t = [torch.from_numpy(a.astype(np.float32)).cuda() for a in (f, x)]
    return [a.to(DT[dt]) for a in t] + [torch.from_numpy(h0.astype(np.float32)).cuda()]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,B,D", [(1, 2, 33), (7, 1, 64), (300, 2, 40), (3000, 1, 66), (700, 13, 1000)])
def test_gated_values_whose_difference_leaves_float32(T, B, D, dt):
    """A logit gate's h lies between its state and x, finite where those are; an
    infinite logit passes the one as it is and nothing of the other."""
    f, x, h0 = _huge(T, B, D, dt, T)
    h, hT = g.gated_fwd(f, x, h0)
    rh, rT, eh, eT = gated_ref.gated(_np(f), _np(x), _np(h0), "logit")
    _within("h", h, rh, eh, dt)
    _within("hT", hT, rT, eT)
    begin = f == -float("inf")
    assert torch.equal(h[begin], x[begin])
    if T == 1:
        y, S = g.gated_step(f, x, h0.clone())
        _within("step", y, rh, eh, dt)
        _within("state", S, rT, eT)
    rng = np.random.default_rng(1)
    dh = torch.from_numpy((1e-3 * rng.standard_normal((T, B, D))).astype(np.float32)).cuda().to(DT[dt])
    r = g.gated_bwd(f, x, h, dh, h0)
    ref, bound = gated_ref.gated_grad(_np(f), _np(x), _np(h), _np(dh), _np(h0), None, "logit")
    for k in ref:
        _within(k, r[k], ref[k], bound[k], dt if k != "dh0" else "f32")


def test_clip_outputs_next_to_each_other():
    """Tensors and outputs that touch are apart; those that overlap are refused."""
    big = torch.randn(40000, device="cuda")
    keep = big.clone()
    cut = [100 * i + (i * i) % 100 for i in range(331)]
    for count in (5, 330):
        big.copy_(keep)
        parts = [big[lo:hi] for lo, hi in zip(cut[:count], cut[1:])]
        norm, ref = gated_ref.clip([_np(t) for t in parts], 1.0)
        g.clip_grads(parts, 1.0)
        for o, r in zip(parts, ref):
            assert (np.abs(_np(o) - r) <= 4 * U * np.abs(r)).all()
        assert torch.equal(big[cut[count]:], keep[cut[count]:])
    a, b = keep[:100], keep[100:200]
    out = torch.full((200,), 7.0, device="cuda")
    for grads, to in (([a, b], [b, a]), ([a, b], [a, a]), ([a, b], [out[:100], out[99:199]]),
                      ([a, b], [out[:100], keep[150:250]]), ([a], [keep[1:101]])):
        with pytest.raises(ValueError):
            g.clip_grads(grads, 1.0, out=to)
    with pytest.raises(ValueError):
        g.clip_grads([a, keep[99:150]], 1.0)
    with pytest.raises(ValueError):
        g.clip_grads([a, b], 1.0, norm=keep[5])
    assert (out == 7.0).all()
    # what is only read may overlap, and a norm is of any list
    g.clip_grads([a, keep[50:150]], 1.0, out=[out[:100], out[100:]])
    norm, ref = gated_ref.clip([_np(a), _np(keep[50:150])], 1.0)
    assert (np.abs(_np(out) - np.concatenate(ref)) <= 4 * U * np.abs(np.concatenate(ref))).all()
    assert abs(g.grad_norm([a, a, keep[50:150]]).item() - np.sqrt(norm ** 2 + (_np(a) ** 2).sum())) <= 4 * U * norm * 2


@pytest.mark.parametrize("K,B,V", [(0, 3, 50), (4, 1, 32000), (2, 400, 9001), (0, 400, 9001)])
def test_verify_status(K, B, V, monkeypatch):
    """The workspace reports the call that used it last, whatever it held.  With one
    poll allowed (set from the host) a sum that is still on its way gives -1 and a
    status; one that is there gives the token."""
    gen = torch.Generator(device="cuda").manual_seed(V)
    x = 2.0 * torch.randn((K + 1, B, V), generator=gen, device="cuda")
    y = 2.0 * torch.randn((K, B, V), generator=gen, device="cuda")
    d = torch.randint(0, V, (K, B), generator=gen, device="cuda")
    u = torch.rand((K + 1, B), generator=gen, device="cuda")
    n = g.workspace_size_verify(K, B, V)
    for q in (y, None):
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        want, acc = g.verify_drafts(x, d, u, q, ws=ws)
        assert g.workspace_status(ws) == g.RNN_OK
        rt, ra = gated_ref.verify(_np(x), d.cpu().numpy(), _np(u), None if q is None else _np(q))
        assert np.array_equal(want.cpu().numpy(), rt) and np.array_equal(acc.cpu().numpy(), ra)
        monkeypatch.setenv("RNN355_SPIN_LIMIT", "1")
        tokens, acc1 = g.verify_drafts(x, d, u, q, ws=ws)
        status = g.workspace_status(ws)
        monkeypatch.delenv("RNN355_SPIN_LIMIT")
        lost = tokens != want
        assert torch.equal(acc, acc1) and (tokens[lost] == -1).all()
        assert status == (g.RNN_ERR_BARRIER_TIMEOUT if lost.any() else g.RNN_OK)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V", [50, 5001, 70001])
def test_verify_equal_rows_that_start_elsewhere(V, dt):
    """The same distribution twice, the draft's rows at another place of their 16
    bytes: nothing is left of the difference, and p itself is drawn from, where a
    draft is refused that has no probability in either, or is outside."""
    K, B = 2, 60
    rng = np.random.default_rng(V)
    x = torch.from_numpy((2.0 * rng.standard_normal((K + 1, B, V))).astype(np.float32)).to(DT[dt]).cuda()
    d = torch.from_numpy(rng.integers(0, V, (K, B))).cuda()
    u = torch.from_numpy(rng.random((K + 1, B)).astype(np.float32)).cuda()
    d[:, ::2] = -1
    bidx = torch.arange(1, B, 2, device="cuda")
    x[0, bidx, d[0, bidx]] = -float("inf")
    for pad in ((3, 0), (1, 4), (0, 1)):
        y = torch.nn.functional.pad(x[:K], pad)[..., pad[0]:pad[0] + V]
        tokens, acc = g.verify_drafts(x, d, u, y)
        rt, ra = gated_ref.verify(_np(x), d.cpu().numpy(), _np(u), _np(y))
        assert not ra.any() and np.array_equal(acc.cpu().numpy(), ra)
        assert np.array_equal(tokens.cpu().numpy(), rt)
        want, _ = g.verify_drafts(x[:1], None, u[K:])
        assert torch.equal(tokens[:1], want)


@pytest.mark.parametrize("sizes", [[(777,), (31,)], [(300000,), (1,), (70000, 3)]], ids=str)
def test_clip_bound_keeps_its_bits(sizes):
    """The bound is taken in 64 bits as it is given: a float32 result is off by its
    own rounding alone, half a step, and a bound past float32 clips."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    grads = [torch.randn(n, generator=gen, device="cuda") for n in sizes]
    for bound in (0.1, 1.0 / 3.0, 1e-4 * np.pi):
        norm, ref = gated_ref.clip([_np(t) for t in grads], bound)
        out = [torch.empty_like(t) for t in grads]
        g.clip_grads(grads, bound, out=out)
        for o, r in zip(out, ref):
            # the sum's, the root's and the factor's 64-bit roundings: below 1e-12
            assert (np.abs(_np(o) - r) <= (U + 1e-12) * np.abs(r) + 1e-45).all(), bound
    t = torch.full((300,), 3e38, device="cuda")
    g.clip_grads([t], 1e39)
    want = 1e39 / np.sqrt(300)
    assert (np.abs(_np(t) - want) <= (U + 1e-12) * want).all()


@pytest.mark.parametrize("n", [4, 1 << 20])
def test_clip_bf16_next_to_a_midpoint(n):
    """Ones of norm sqrt(n), clipped so that the result lies 2^-30 to either side of
    the middle of two bf16 numbers: the nearer one, whichever is even."""
    for k in (1, 2):
        mid = 0.5 + (k + 0.5) * 2.0 ** -8
        for off, want in ((-2.0 ** -30, 0.5 + k * 2.0 ** -8), (2.0 ** -30, 0.5 + (k + 1) * 2.0 ** -8)):
            t = torch.ones(n, dtype=torch.bfloat16, device="cuda")
            out = torch.empty_like(t)
            g.clip_grads([t], float(np.sqrt(n)) * (mid + off), out=[out])
            assert (out.double() == want).all(), (k, off, out[0].item())


def test_clip_bf16_rounds_once():
    """Random values and bounds against the 64-bit product rounded to bf16 once, bit for
    bit (the product is off by less than 2^-45 of itself: one border in 10^10 values)."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    t = torch.randn(40001, generator=gen, device="cuda").bfloat16()
    v, out = _np(t), torch.empty_like(t)
    norm = float(np.sqrt((v ** 2).sum()))
    for share in np.random.default_rng(3).uniform(0.1, 1.0, 40):
        g.clip_grads([t], share * norm, out=[out])
        m, e = np.frexp(v * (share * norm / norm))  # |m| in [1/2, 1): eight bits of it
        assert np.array_equal(_np(out), np.ldexp(np.rint(m * 256.0), e - 8)), share


def test_gated_states_that_start_elsewhere_are_refused_by_name():
    f, x, dh = (torch.randn((1, 1, 129), device="cuda") for _ in range(3))
    s = torch.randn((2, 129), device="cuda")[1:]
    for call, name in ((lambda: g.gated_fwd(f, x, s), "h0"), (lambda: g.gated_fwd(f, x, out={"hT": s}), "hT"),
                       (lambda: g.gated_step(f, x, s), "h"), (lambda: g.gated_step(f, x, s.clone(), h_out=s), "h_out"),
                       (lambda: g.gated_bwd(f, x, x, dh, s), "h0"), (lambda: g.gated_bwd(f, x, x, dh, None, s), "dhT"),
                       (lambda: g.gated_bwd(f, x, x, dh, out={"dh0": s}), "dh0")):
        with pytest.raises(ValueError, match=name + " must start"):
            call()
    # what is read value by value may start anywhere
    logits = torch.randn((1, 3, 50), device="cuda")
    u, t = torch.rand((2, 3), device="cuda"), torch.rand(4, device="cuda") + 0.5
    tokens, _ = g.verify_drafts(logits, None, u[1:], temperature=t[1:])
    want, _ = g.verify_drafts(logits, None, u[1:].clone(), temperature=t[1:].clone())
    assert torch.equal(tokens, want)


def test_gated_smaller_side_of_the_gate():
    """Read from one step: a itself of a state of 1 and an x of 0 where the gate is shut,
    1 - a of an x of 1 and a state of 0 where it is open, against sigmoid in 64 bits."""
    v = np.concatenate([np.linspace(0.0, 87.2, 200001), 2.0 ** np.arange(-20.0, 0.0)])
    v = torch.from_numpy(v.astype(np.float32)).cuda()[None, None]
    zero, one = torch.zeros_like(v), torch.ones_like(v)
    ref = np.exp(-_np(v)) / (1.0 + np.exp(-_np(v)))
    for f, x, h0 in ((-v, zero, one[0]), (v, one, zero[0])):
        err = np.abs(_np(g.gated_step(f, x, h0.clone())[0]) - ref)
        assert (err <= (2 * _np(v) + 6) * U * ref).all()


@pytest.mark.parametrize("gate", ["logit", "decay"])
@pytest.mark.parametrize("T,B,D", [(6000, 4, 258), (20011, 1, 129)])
def test_gated_many_segments_bound_carried(T, B, D, gate):
    """Long float32 sequences within the bounds that gated_ref derives, carried along
    the 64-bit definition on the device step by step."""
    gen = torch.Generator(device="cuda").manual_seed(T)
    f = torch.randn((T, B, D), generator=gen, device="cuda") + 3.0
    f = f if gate == "logit" else torch.sigmoid(f)
    x, dh = (torch.randn((T, B, D), generator=gen, device="cuda") for _ in range(2))
    h0, dhT = (torch.randn((B, D), generator=gen, device="cuda") for _ in range(2))
    h, hT = g.gated_fwd(f, x, h0, gate=gate)
    r = g.gated_bwd(f, x, h, dh, h0, dhT, gate=gate)
    fd = f.double()
    if gate == "logit":
        a, s = torch.sigmoid(fd), torch.sigmoid(-fd)
        w = (2 * fd.abs() + 7) * torch.minimum(a, s)
    else:
        a, s, w = fd, torch.ones_like(fd), torch.zeros_like(fd)
    ok = torch.ones((), dtype=torch.bool, device="cuda")
    S, M, E = h0.double(), h0.double().abs(), torch.zeros((B, D), dtype=torch.float64, device="cuda")
    for t in range(T):
        xt = x[t].double()
        m = a[t] * M + s[t] * xt.abs()
        E = a[t] * E + U * (w[t] * (xt.abs() + M) + 4 * m)
        S, M = a[t] * S + s[t] * xt, m
        ok &= ((h[t] - S).abs() <= E).all()
    assert ok and ((hT - S).abs() <= E).all()
    e, m, E = dhT.double(), dhT.double().abs(), torch.zeros_like(S)
    af = fd.abs() if gate == "logit" else torch.zeros_like(fd)
    for t in range(T - 1, -1, -1):
        gt, mg = e + dh[t].double(), m + dh[t].double().abs()
        Eg = E + U * mg
        bx = s[t] * (Eg + U * (2 * af[t] + 8) * mg) if gate == "logit" else Eg
        ok &= ((r["dx"][t] - s[t] * gt).abs() <= bx).all()
        before = h[t - 1].double() if t else h0.double()
        if gate == "logit":
            w2, df = a[t] * s[t], gt * (before - x[t].double()) * a[t] * s[t]
            bf = w2 * (before.abs() + x[t].double().abs()) * (Eg + U * (4 * af[t] + 16) * mg)
        else:
            df, bf = gt * before, before.abs() * (Eg + U * mg)
        ok &= ((r["df"][t] - df).abs() <= bf).all()
        E = a[t] * Eg + U * (w[t] + 4 * a[t]) * mg
        e, m = a[t] * gt, a[t] * mg
    assert ok and ((r["dh0"] - e).abs() <= E).all()
