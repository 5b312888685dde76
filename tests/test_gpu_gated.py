"""The gated linear recurrence against its 64-bit definition, elementwise, within
the bounds that gated_ref derives; bf16 outputs add half their spacing."""
import numpy as np
import pytest

from tests import gated_ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gru_recurrence_amd as g  # noqa: E402

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
TINY = 1e-37  # values near the smallest normal float32 may be flushed


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _rand(rng, shape, dt, std=1.0):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * std).to(DT[dt]).cuda()


def _within(name, y, ref, bound, dt="f32"):
    y = _np(y) if torch.is_tensor(y) else y
    assert y.shape == ref.shape, (name, y.shape, ref.shape)
    assert np.isfinite(y).all(), name
    err = np.abs(y - ref)
    limit = bound + TINY
    if dt == "bf16":
        limit = limit + 2.0 ** -8 * (np.abs(ref) + bound)
    over = err > limit
    assert not over.any(), (name, int(over.sum()), float(err.max()), np.argwhere(over)[:3].tolist())


def _view(t, layout):
    """The same values under other strides."""
    T, B, D = t.shape
    if layout == "bt":
        return t.transpose(0, 1).contiguous().transpose(0, 1)
    if layout == "odd":      # rows that start at an odd element, of odd stride
        return torch.nn.functional.pad(t, (1, 2 + D % 2))[..., 1:D + 1]
    if layout == "fused":    # the second half of a projection
        return torch.cat([t, t], -1)[..., D:]
    return t


def _case(seed, T, B, D, dt, gate, layout="dense", ragged=False):
    rng = np.random.default_rng(seed)
    if gate == "logit":
        f = 3.0 * rng.standard_normal((T, B, D)) + rng.choice([-2.0, 2.0, 6.0], (D,))
    else:
        f = 1.0 - np.exp(rng.uniform(np.log(1e-3), 0.0, (T, B, D)))
        f *= rng.choice([1.0, 1.0, 1.0, -1.0], (T, B, D))
        f[rng.random((T, B, D)) < 0.02] = 0.0
        f[rng.random((T, B, D)) < 0.02] = 1.0
    f = torch.from_numpy(f.astype(np.float32)).to(DT[dt]).cuda()
    x, dh = _rand(rng, (T, B, D), dt), _rand(rng, (T, B, D), dt)
    h0, dhT = _rand(rng, (B, D), "f32"), _rand(rng, (B, D), "f32")
    lens = None
    if ragged:
        lens = rng.integers(0, T + 1, B)
        lens[0] = 0
        lens[-1] = T if B > 1 else T // 2
        lens = torch.from_numpy(lens.astype(np.int32)).cuda()
    return [_view(t, layout) for t in (f, x, dh)] + [h0, dhT, lens]


def _check(T, B, D, dt, gate, layout="dense", ragged=False, state=True, seed=0):
    f, x, dh, h0, dhT, lens = _case(seed + T + D, T, B, D, dt, gate, layout, ragged)
    if not state:
        h0 = dhT = None
    h, hT = g.gated_fwd(f, x, h0, gate=gate, lens=lens)
    assert h.dtype == f.dtype and hT.dtype == torch.float32
    n = None if lens is None else lens.cpu().numpy()
    rh, rT, eh, eT = gated_ref.gated(_np(f), _np(x), _np(h0), gate, n)
    _within("h", h, rh, eh, dt)
    _within("hT", hT, rT, eT)
    h = _view(h, layout)
    r = g.gated_bwd(f, x, h, dh, h0, dhT, gate=gate, lens=lens)
    ref, bound = gated_ref.gated_grad(_np(f), _np(x), _np(h), _np(dh), _np(h0), _np(dhT), gate, n)
    for k in ("df", "dx"):
        assert r[k].dtype == f.dtype
        _within(k, r[k], ref[k], bound[k], dt)
    _within("dh0", r["dh0"], ref["dh0"], bound["dh0"])


@pytest.mark.parametrize("gate", ["logit", "decay"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,B,D", [
    (1, 1, 1), (2, 1, 2), (3, 2, 7), (7, 1, 64), (8, 3, 65), (16, 1, 128), (63, 2, 33), (64, 1, 256),
    (65, 5, 100), (127, 1, 130), (128, 2, 66), (129, 1, 512), (257, 3, 21), (1000, 1, 40), (2049, 2, 5),
    (5000, 1, 2), (333, 40, 17)])
def test_gated(T, B, D, dt, gate):
    _check(T, B, D, dt, gate)


@pytest.mark.parametrize("gate", ["logit", "decay"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["fused", "bt", "odd"])
def test_gated_layouts(layout, dt, gate):
    _check(150, 3, 64, dt, gate, layout)
    _check(70, 2, 37, dt, gate, layout, state=False)
    _check(700, 2, 30, dt, gate, layout, ragged=True)


@pytest.mark.parametrize("gate", ["logit", "decay"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,B,D", [(1, 4, 6), (5, 1, 64), (100, 5, 33), (400, 7, 64), (1500, 9, 10)])
def test_gated_ragged(T, B, D, dt, gate):
    _check(T, B, D, dt, gate, ragged=True)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gated_without_state(dt):
    _check(300, 2, 48, dt, "logit", state=False)
    _check(1, 3, 9, dt, "decay", state=False)


@pytest.mark.parametrize("gate", ["logit", "decay"])
@pytest.mark.parametrize("T,B,D,layout,ragged", [(300, 10, 1024, "fused", True), (512, 21, 500, "bt", False),
                                                 (700, 13, 1000, "dense", True), (1024, 11, 932, "dense", False)])
def test_gated_many_channels(T, B, D, layout, ragged, gate):
    """Many channels of some hundred steps each; a last state written over the first."""
    f, x, _, h0, _, lens = _case(T, T, B, D, "bf16", gate, layout, ragged)
    n = None if lens is None else lens.cpu().numpy()
    rh, rT, eh, eT = gated_ref.gated(_np(f), _np(x), _np(h0), gate, n)
    h, hT = g.gated_fwd(f, x, h0, gate=gate, lens=lens)
    _within("h", h, rh, eh, "bf16")
    _within("hT", hT, rT, eT)
    h1, _ = g.gated_fwd(f, x, h0, gate=gate, lens=lens, out={"hT": h0})
    assert torch.equal(h1, h) and torch.equal(h0, hT)


@pytest.mark.parametrize("gate", ["logit", "decay"])
@pytest.mark.parametrize("T,B,D", [(40000, 1, 70), (9000, 4, 258), (20011, 1, 129)])
def test_gated_many_segments(T, B, D, gate):
    """Long sequences, against the definition in 64 bits on the device."""
    gen = torch.Generator(device="cuda").manual_seed(T)
    f = torch.randn((T, B, D), generator=gen, device="cuda") + 3.0
    f = f if gate == "logit" else torch.sigmoid(f)
    x, dh = (torch.randn((T, B, D), generator=gen, device="cuda") for _ in range(2))
    h0, dhT = (torch.randn((B, D), generator=gen, device="cuda") for _ in range(2))
    h, hT = g.gated_fwd(f, x, h0, gate=gate)
    r = g.gated_bwd(f, x, h, dh, h0, dhT, gate=gate)
    fd = f.double()
    a, s = (torch.sigmoid(fd), torch.sigmoid(-fd)) if gate == "logit" else (fd, torch.ones_like(fd))
    S, m = h0.double(), h0.double().abs()
    worst = 0.0
    for t in range(T):
        S = a[t] * S + s[t] * x[t].double()
        m = a[t] * m + s[t] * x[t].double().abs()
        if t % 97 == 0 or t == T - 1:
            # sums of magnitudes m, each step's roundings forgotten at a's pace: at most
            # 4 u m / (1 - a), and 1 / (1 - a) stays below 2000 here (f < 7.6)
            worst = max(worst, ((h[t] - S).abs() / m).max().item())
    assert worst <= 4 * 2000 * 2.0 ** -24, worst
    assert ((hT - S).abs() <= 4 * 2000 * 2.0 ** -24 * m).all()
    e, me = dhT.double(), dhT.double().abs()
    worst = 0.0
    for t in range(T - 1, -1, -1):
        gt, mg = e + dh[t].double(), me + dh[t].double().abs()
        if t % 97 == 0:
            worst = max(worst, ((r["dx"][t] - s[t] * gt).abs() / (s[t] * mg)).max().item())
        e, me = a[t] * gt, a[t] * mg
    assert worst <= 4 * 2000 * 2.0 ** -24, worst
    assert ((r["dh0"] - e).abs() <= 4 * 2000 * 2.0 ** -24 * me).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gated_outputs_as_views(dt):
    """h and the gradients written into halves of larger arrays, batch-first ones,
    and rows that start at an odd element; nothing else is touched."""
    T, B, D = 200, 3, 50
    f, x, dh, h0, dhT, lens = _case(5, T, B, D, dt, "logit", ragged=True)
    h, _ = g.gated_fwd(f, x, h0, lens=lens)
    want = g.gated_bwd(f, x, h, dh, h0, dhT, lens=lens)
    big = torch.full((T, B, 2 * D + 3), 7.0, dtype=DT[dt], device="cuda")
    for lo in (0, 1, 3):
        big.fill_(7.0)
        o = big[..., lo:lo + D]
        r, _ = g.gated_fwd(f, x, h0, lens=lens, out={"h": o})
        assert r is o and torch.equal(o, h)
        assert (big[..., :lo] == 7).all() and (big[..., lo + D:] == 7).all()
    big.fill_(7.0)
    out = {"df": big[..., :D], "dx": big[..., D:2 * D]}
    r = g.gated_bwd(f, x, h, dh, h0, dhT, lens=lens, out=out)
    for k in ("df", "dx"):
        assert r[k] is out[k] and torch.equal(out[k], want[k])
    assert (big[..., 2 * D:] == 7).all()
    bt = torch.empty((B, T, D), dtype=DT[dt], device="cuda").transpose(0, 1)
    g.gated_fwd(f, x, h0, lens=lens, out={"h": bt})
    assert torch.equal(bt, h)


@pytest.mark.parametrize("gate", ["logit", "decay"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,D", [(1, 1), (3, 65), (64, 128), (5, 514)])
def test_gated_step(B, D, dt, gate):
    """Token by token equals the definition; in place and to another state."""
    T = 5
    f, x, _, h0, _, _ = _case(B + D, T, B, D, dt, gate, "fused")
    rh, rT, eh, eT = gated_ref.gated(_np(f), _np(x), _np(h0), gate)
    keep, S = h0.clone(), h0
    for t in range(T):
        to = torch.empty_like(S) if t == 0 else None
        y, S2 = g.gated_step(f[t:t + 1], x[t:t + 1], S, gate=gate, h_out=to)
        assert (S2 is S) == (t > 0) and tuple(y.shape) == (1, B, D)
        S = S2
        _within("y", y[0], rh[t], eh[t], dt)
    assert torch.equal(h0, keep)
    _within("state", S, rT, eT)


def test_gated_prompt_then_steps():
    f, x, _, h0, _, _ = _case(2, 300, 2, 96, "f32", "logit")
    h, hT = g.gated_fwd(f, x, h0)
    part, S = g.gated_fwd(f[:290], x[:290], h0)
    rows = [part]
    for t in range(290, 300):
        rows.append(g.gated_step(f[t:t + 1], x[t:t + 1], S)[0])
    assert (torch.cat(rows) - h).norm() <= 1e-6 * h.norm()
    assert (S - hT).norm() <= 1e-6 * hT.norm()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 50, 1200, 20000])
def test_gated_state_in_place(T, dt):
    """The last state over the first, forward and backward, where the sequence
    runs in segments at once: the same bits as into another tensor, every time."""
    f, x, dh, h0, dhT, _ = _case(T, T, 2, 66, dt, "logit")
    h, hT = g.gated_fwd(f, x, h0)
    r = g.gated_bwd(f, x, h, dh, h0, dhT)
    for _ in range(3):
        S, E = h0.clone(), dhT.clone()
        h1, S1 = g.gated_fwd(f, x, S, out={"hT": S})
        assert S1 is S and torch.equal(S, hT) and torch.equal(h1, h)
        r1 = g.gated_bwd(f, x, h, dh, h0, E, out={"dh0": E})
        assert r1["dh0"] is E
        for k in r:
            assert torch.equal(r1[k], r[k]), k


def test_gated_lens_are_prefixes():
    """The state after lens tokens is that of a call on those alone; lens outside
    [0, T] are its nearest end; what stands behind is not read."""
    T, B, D = 130, 6, 64
    f, x, dh, h0, dhT, _ = _case(3, T, B, D, "f32", "logit")
    lens = torch.tensor([-5, 0, 1, 64, 130, 1000], dtype=torch.int32, device="cuda")
    f2, x2, dh2 = f.clone(), x.clone(), dh.clone()
    for b, n in enumerate(lens.clamp(0, T).tolist()):
        for t in (f2, x2, dh2):
            t[n:, b] = float("nan")
    h, hT = g.gated_fwd(f2, x2, h0, lens=lens)
    r = g.gated_bwd(f2, x2, h, dh2, h0, dhT, lens=lens)
    for b, n in enumerate(lens.clamp(0, T).tolist()):
        one = slice(b, b + 1)
        assert not h[n:, b].any() and not r["df"][n:, b].any() and not r["dx"][n:, b].any()
        if n == 0:
            assert torch.equal(hT[b], h0[b]) and torch.equal(r["dh0"][b], dhT[b])
            continue
        h1, S1 = g.gated_fwd(f[:n, one], x[:n, one], h0[one].contiguous())
        assert (h[:n, one] - h1).abs().max() <= 1e-5 and (hT[one] - S1).abs().max() <= 1e-5
        r1 = g.gated_bwd(f[:n, one], x[:n, one], h1, dh[:n, one], h0[one].contiguous(),
                         dhT[one].contiguous())
        for k in ("df", "dx"):
            assert (r[k][:n, one] - r1[k]).abs().max() <= 1e-4, k
        assert (r["dh0"][one] - r1["dh0"]).abs().max() <= 1e-4


def test_gated_extreme_gates():
    """Gates shut and open for good: no NaN, the closed forms."""
    T, B, D = 300, 1, 8
    x = torch.randn((T, B, D), device="cuda")
    h0 = torch.randn((B, D), device="cuda")
    inf = float("inf")
    for v, want, last in ((-inf, x, x[-1]), (-200.0, x, x[-1]),
                          (inf, h0.expand(T, B, D), h0), (200.0, h0.expand(T, B, D), h0)):
        f = torch.full((T, B, D), v, device="cuda")
        h, hT = g.gated_fwd(f, x, h0)
        assert torch.equal(h, want.contiguous()) and torch.equal(hT, last)
        r = g.gated_bwd(f, x, h, torch.ones_like(x), h0, None)
        for k in r:
            assert torch.isfinite(r[k]).all(), (v, k)
        shut = v < 0
        assert torch.equal(r["dx"], torch.full_like(x, 1.0 if shut else 0.0)), v
        assert (r["df"].abs() <= 1e-30).all()
        assert torch.equal(r["dh0"], torch.full_like(h0, 0.0 if shut else T)), v
    # products of decays that leave float32 at the small end, and states of zero
    f = torch.full((T, B, D), 1e-3, device="cuda")
    h, hT = g.gated_fwd(f, torch.zeros_like(x), h0, gate="decay")
    assert not hT.any() and torch.isfinite(h).all()
    h, hT = g.gated_fwd(torch.ones_like(f), torch.ones_like(f), None, gate="decay")
    assert torch.equal(h[:, 0, 0], torch.arange(1.0, T + 1, device="cuda"))


@pytest.mark.parametrize("T,D", [(1, 64), (5, 130), (300, 40), (3000, 70), (600, 2048)])
def test_gated_nearly_shut_gates(T, D):
    """Gates of 1e-7 to 1e-4 between large and small values, a gradient from the last
    token alone: what they let through is right relative to itself."""
    rng = np.random.default_rng(T)
    f = 3.0 * rng.standard_normal((T, 1, D)) + 3.0
    low = rng.random(f.shape) < 0.05
    low[0] = True
    f[low] = -rng.uniform(9.0, 16.0, low.sum())
    x = np.abs(rng.standard_normal(f.shape)) * 10.0 ** rng.integers(-4, 5, f.shape)
    dh = np.zeros(f.shape)
    dh[-1] = rng.standard_normal((1, D))
    f, x, dh = (torch.from_numpy(t.astype(np.float32)).cuda() for t in (f, x, dh))
    h0 = torch.full((1, D), 1e6, device="cuda")
    h, hT = g.gated_fwd(f, x, h0)
    rh, rT, eh, eT = gated_ref.gated(_np(f), _np(x), _np(h0), "logit")
    _within("h", h, rh, eh)
    _within("hT", hT, rT, eT)
    if T == 1:
        y, _ = g.gated_step(f, x, h0.clone())
        _within("step", y, rh, eh)
    r = g.gated_bwd(f, x, h, dh, h0)
    ref, bound = gated_ref.gated_grad(_np(f), _np(x), _np(h), _np(dh), _np(h0), None, "logit")
    for k in ref:
        _within(k, r[k], ref[k], bound[k])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,B,D", [(7, 2, 33), (500, 3, 64), (2500, 1, 66), (900, 16, 1024)])
def test_gated_logits_of_minus_infinity_begin_a_sequence(T, B, D, dt):
    """Sequences packed along time: nothing passes from one to the next."""
    rng = np.random.default_rng(T)
    f, x, dh = (_rand(rng, (T, B, D), dt) for _ in range(3))
    at = T // 2
    x[:at] *= 1e6
    f[at] = -float("inf")
    h, hT = g.gated_fwd(f, x)
    assert torch.equal(h[at], x[at])
    h1, hT1 = g.gated_fwd(f[at:], x[at:])
    n = [_np(t[at:]) for t in (f, x)]
    rh, rT, eh, eT = gated_ref.gated(*n, None, "logit")
    for y, yT in ((h[at:], hT), (h1, hT1)):
        _within("h", y, rh, eh, dt)
        _within("hT", yT, rT, eT)
    dh[:at] = 0.0
    r = g.gated_bwd(f, x, h, dh)
    assert not r["dx"][:at].any() and not r["df"][:at].any() and not r["dh0"].any()


def test_gated_nan_stays_in_its_channel_and_future():
    f, x, _, h0, _, _ = _case(8, 700, 2, 66, "f32", "logit")
    want, _ = g.gated_fwd(f, x, h0)
    x[300, 1, 17] = float("nan")
    h, hT = g.gated_fwd(f, x, h0)
    bad = torch.isnan(h)
    assert bad[300:, 1, 17].all() and bad.sum() == 400 and torch.isnan(hT).sum() == 1
    assert torch.equal(h[~bad], want[~bad])


def test_gated_strides_past_32_bits():
    f, x, dh, h0, dhT, _ = _case(6, 3, 2, 64, "bf16", "logit")
    far = torch.empty((3, 1 << 30), dtype=torch.bfloat16, device="cuda")
    ff = far[:, 128:256].view(3, 2, 64)
    ff.copy_(f)
    h, hT = g.gated_fwd(f, x, h0)
    h1, S1 = g.gated_fwd(ff, x, h0)
    assert torch.equal(h, h1) and torch.equal(hT, S1)
    r, r1 = g.gated_bwd(f, x, h, dh, h0, dhT), g.gated_bwd(ff, x, h, dh, h0, dhT)
    for k in r:
        assert torch.equal(r[k], r1[k])


def test_gated_offsets_past_32_bits():
    """2.5e9 values: some rows against calls on those alone, which are cut the same
    way, so that their sums run in the same order."""
    T, B, D = 300, 128, 65536
    gen = torch.Generator(device="cuda").manual_seed(0)
    f, x = (torch.empty((T, B, D), dtype=torch.bfloat16, device="cuda").normal_(generator=gen) for _ in range(2))
    h, hT = g.gated_fwd(f, x)
    r = g.gated_bwd(f, x, h, x)
    for b in (0, 60, 120):
        rows = slice(b, b + 8)
        cut = [t[:, rows].contiguous() for t in (f, x)]
        h1, S1 = g.gated_fwd(*cut)
        assert torch.equal(h[:, rows], h1) and torch.equal(hT[rows], S1)
        r1 = g.gated_bwd(*cut, h1, cut[1])
        for k in ("df", "dx"):
            assert torch.equal(r[k][:, rows], r1[k]), k
        assert torch.equal(r["dh0"][rows], r1["dh0"])


@pytest.mark.parametrize("D,layout", [(258, "fused"), (257, "dense")])
def test_gated_many_values_bf16(D, layout):
    """A call of many workgroups, with and without pairs of channels, against the
    definition in 64 bits on the device: bounds as in gated_ref, where a step's share
    u ((2 |f| + 7) s (|x| + M) + 4 M) stays below 16 u M' with M' = M + s |x| (|f| < 9,
    s (2 |f| + 7) < 9), and the sum over steps forgets at a's pace: carried along."""
    T, B = 4200, 16
    gen = torch.Generator(device="cuda").manual_seed(D)
    f = (torch.randn((T, B, D), generator=gen, device="cuda") + 2.0).bfloat16()
    x, dh = (torch.randn((T, B, D), generator=gen, device="cuda").bfloat16() for _ in range(2))
    h0, dhT = (torch.randn((B, D), generator=gen, device="cuda") for _ in range(2))
    f, x, dh = (_view(t, layout) for t in (f, x, dh))
    assert f.float().abs().max() < 9
    h, hT = g.gated_fwd(f, x, h0)
    r = g.gated_bwd(f, x, h, dh, h0, dhT)
    a, s = torch.sigmoid(f.double()), torch.sigmoid(-f.double())
    u, S, M = 2.0 ** -24, h0.double(), h0.double().abs()
    E = torch.zeros_like(S)
    ok = torch.ones((), dtype=torch.bool, device="cuda")
    for t in range(T):
        xt = x[t].double()
        S, M = a[t] * S + s[t] * xt, a[t] * M + s[t] * xt.abs()
        E = a[t] * E + 16 * u * (M + s[t] * xt.abs())
        ok &= ((h[t].double() - S).abs() <= E + 2.0 ** -8 * (S.abs() + E)).all()
    assert ok and ((hT - S).abs() <= E).all()
    e, m, E = dhT.double(), dhT.double().abs(), torch.zeros_like(S)
    for t in range(T - 1, -1, -1):
        gt, mt, Et = e + dh[t].double(), m + dh[t].double().abs(), E
        Et = Et + u * mt
        dx, bx = s[t] * gt, s[t] * (Et + 26 * u * mt)
        ok &= ((r["dx"][t].double() - dx).abs() <= bx + 2.0 ** -8 * (dx.abs() + bx)).all()
        e, m, E = a[t] * gt, a[t] * mt, a[t] * Et + 16 * u * mt
    assert ok and ((r["dh0"] - e).abs() <= E).all()


def test_gated_inputs_shared_by_the_batch():
    """f and x broadcast over the batch (stride 0)."""
    f, x, dh, h0, dhT, _ = _case(2, 90, 4, 32, "f32", "logit")
    f1, x1 = f[:, :1].expand(-1, 4, -1), x[:, :1].expand(-1, 4, -1)
    h, hT = g.gated_fwd(f1, x1, h0)
    h2, hT2 = g.gated_fwd(f1.contiguous(), x1.contiguous(), h0)
    assert torch.equal(h, h2) and torch.equal(hT, hT2)
    a = g.gated_bwd(f1, x1, h, dh, h0, dhT)
    b = g.gated_bwd(f1.contiguous(), x1.contiguous(), h, dh, h0, dhT)
    for k in a:
        assert torch.equal(a[k], b[k])


@pytest.mark.parametrize("gate", ["logit", "decay"])
def test_gated_gradient_by_differences(gate):
    """Central differences of the 64-bit definition at the library's gradient."""
    f, x, dh, h0, dhT, lens = _case(11, 40, 3, 20, "f32", gate, ragged=True)
    n = lens.cpu().numpy()
    args = {"f": _np(f), "x": _np(x), "h0": _np(h0)}

    def loss(**kw):
        a = {**args, **kw}
        h, S, _, _ = gated_ref.gated(a["f"], a["x"], a["h0"], gate, n)
        return (h * _np(dh)).sum() + (S * _np(dhT)).sum()
    h, _ = g.gated_fwd(f, x, h0, gate=gate, lens=lens)
    r = g.gated_bwd(f, x, h, dh, h0, dhT, gate=gate, lens=lens)
    rng, eps = np.random.default_rng(0), 1e-5
    for k, v in args.items():
        for _ in range(5):
            d = rng.standard_normal(v.shape)
            num = (loss(**{k: v + eps * d}) - loss(**{k: v - eps * d})) / (2 * eps)
            grad = _np(r["d" + k]) * d
            # the gradient's float32 roundings, and eps^2 of the third derivative
            assert abs(num - grad.sum()) <= 1e-5 * np.abs(grad).sum() + 1e-7, k


def test_gated_on_another_stream_and_captured():
    f, x, dh, h0, dhT, lens = _case(4, 3000, 3, 65, "bf16", "logit", ragged=True)
    d = g.GatedDims(3000, 3, 65)
    u8 = lambda n: torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")  # noqa: E731
    w = [u8(g.workspace_size_gated(op, d, g.RNN_BF16)) for op in (g.OP_GATED_FWD, g.OP_GATED_BWD)]

    def calls(**kw):
        h, hT = g.gated_fwd(f, x, h0, lens=lens, **({"ws": w[0]} if not kw else kw))
        r = g.gated_bwd(f, x, h, dh, h0, dhT, lens=lens, **({"ws": w[1]} if not kw else kw))
        return [h, hT, *r.values()]
    want = calls()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(4):
        side.wait_stream(torch.cuda.current_stream())
        got = calls(stream=side)
        torch.full((1 << 20,), 7.0, device="cuda")
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = calls()
    for i in range(4):
        x.copy_(x.roll(i, 0))
        f.copy_(f.roll(i, 2))
        lens.copy_(lens.roll(1))
        graph.replay()
        got = [t.clone() for t in out]
        for a, b in zip(got, calls()):
            assert torch.equal(a, b), i
        torch.cuda.synchronize()


def test_gated_wait_timeout_is_reported(monkeypatch):
    """With one poll allowed (set from the host) waits between segments give up, the
    kernels end normally and the workspace reports it; the next call clears it."""
    f, x, dh, h0, dhT, _ = _case(1, 60000, 1, 96, "f32", "logit")
    ws = torch.empty(max(g.workspace_size_gated(op, g.GatedDims(60000, 1, 96), g.RNN_F32)
                         for op in (g.OP_GATED_FWD, g.OP_GATED_BWD)), dtype=torch.uint8, device="cuda")
    calls = [lambda: g.gated_fwd(f, x, h0, ws=ws), lambda: g.gated_bwd(f, x, x, dh, h0, dhT, ws=ws)]
    for call in calls:
        monkeypatch.setenv("RNN355_SPIN_LIMIT", "1")
        call()
        assert g.workspace_status(ws) == g.RNN_ERR_BARRIER_TIMEOUT
        monkeypatch.delenv("RNN355_SPIN_LIMIT")
        call()
        assert g.workspace_status(ws) == g.RNN_OK


def test_gated_two_calls_at_once():
    """Calls on two streams, each with its workspace, over and over."""
    cases = [_case(s, 6000, 2, 130, "f32", "logit") for s in (1, 2)]
    want = [g.gated_fwd(c[0], c[1], c[3]) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for _ in range(6):
        for c, s in zip(cases, streams):
            got.append(g.gated_fwd(c[0], c[1], c[3], stream=s))
    torch.cuda.synchronize()
    for i, (h, hT) in enumerate(got):
        assert torch.equal(h, want[i % 2][0]) and torch.equal(hT, want[i % 2][1])
