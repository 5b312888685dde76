"""The operators around the recurrence (embedding, token log probabilities,
linear attention) against their 64-bit definitions (lm_ref), elementwise.

Bounds, u = 2^-24 the float32 rounding unit; rounding to bf16 (8 significant
bits) moves a value by at most half its spacing, r:
  embedding          the float32 product rounded to the type, bit for bit
  embedding gradient n terms added in float32: (n + 2) u sum|terms|
  log probabilities  e^z in float32 has a relative error of about 2|z| u, the
                     sums over a row 48 u (32 in a thread, then a tree), and
                     the final subtraction u (|l| + |lse|).  With |l| <= 40:
                     below 200 u + 40 u = 1.5e-5, taken as 2e-5.  Entropy adds
                     the sum of z e^z, |z| times that: 2e-4 (mean |z| <= 10).
  their gradient     p is off by u (4|lse| + 4|log p| + 16) relative
  linear attention   sums of at most D + T + 64 terms and decays a^n off by
                     2 u |n log2 a| (under 30 where the weight matters):
                     c = (D + T + 64) u + 3e-6 times the sum of magnitudes;
                     bf16 calls add three splits of 2^-17 and the output's r.
"""
import numpy as np
import pytest

from tests import lm_ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gru_recurrence_amd as g  # noqa: E402

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _np(t):
    return t.detach().double().cpu().numpy()


def _rand(rng, shape, dt, std=1.0):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * std).to(DT[dt]).cuda()


def _r(ref, dt):
    """Half the spacing of bf16 numbers at each value; 0 for float32."""
    if dt != "bf16":
        return np.zeros_like(ref)
    a = np.where(np.isfinite(ref), np.abs(ref), 0.0)
    return np.where(a > 0, np.exp2(np.floor(np.log2(np.where(a > 0, a, 1.0))) - 8), 0.0)


def _within(name, y, ref, bound):
    y = _np(y) if torch.is_tensor(y) else y
    assert y.shape == ref.shape, (name, y.shape, ref.shape)
    bad = ~np.isfinite(ref)
    assert np.array_equal(np.isnan(y), np.isnan(ref)), name
    assert np.array_equal(y[bad & ~np.isnan(ref)], ref[bad & ~np.isnan(ref)]), name
    err = np.abs(np.where(bad, 0, y) - np.where(bad, 0, ref))
    over = err > np.broadcast_to(bound, err.shape)
    assert not over.any(), (name, int(over.sum()), float(err.max()))


# -------------------------------------------------------------- embedding
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,B,V,D,order,ids", [
    (1, 1, 1, 1, "tb", "i64"), (1, 3, 7, 8, "tb", "i32"), (5, 4, 100, 64, "bt", "i64"),
    (33, 2, 257, 129, "tb", "i64"), (17, 3, 50, 130, "bt", "i32"), (9, 5, 31, 768, "bt", "i64"),
    (3, 2, 9, 1028, "tb", "i32"), (64, 8, 300, 96, "tb", "i64")])
def test_embed_fwd(T, B, V, D, order, ids, dt):
    rng = np.random.default_rng(T * 1000 + D)
    table = _rand(rng, (V, D), dt)
    n = rng.integers(-2, V + 2, (T, B))  # some outside on either side
    t = torch.from_numpy(n).to(torch.int32 if ids == "i32" else torch.int64).cuda()
    if order == "bt":
        t = t.t().contiguous().t()
        assert B == 1 or T == 1 or not t.is_contiguous()
    x = g.embed_fwd(t, table, 1.7)
    assert x.dtype == table.dtype and tuple(x.shape) == (T, B, D)
    ref = torch.from_numpy(lm_ref.embed(n, _np(table), 1.0)).float() * np.float32(1.7)
    assert torch.equal(x.cpu(), ref.to(DT[dt]))


def test_embed_fwd_table_views():
    """Rows at a stride, a table that starts at an odd element, 1-D ids."""
    rng = np.random.default_rng(3)
    big = _rand(rng, (40, 200), "bf16")
    ids = torch.from_numpy(rng.integers(0, 40, 23)).cuda()
    for lo, hi in ((0, 64), (3, 67), (8, 136), (1, 200), (2, 64)):
        table = big[:, lo:hi]
        x = g.embed_fwd(ids, table)
        assert torch.equal(x, table[ids])
    # a table of more than 2^31 elements apart
    far = torch.empty((3, 1 << 31), dtype=torch.bfloat16, device="cuda")[:, 5:69]
    far.copy_(_rand(rng, (3, 64), "bf16"))
    assert torch.equal(g.embed_fwd(ids % 3, far), far[ids % 3])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,B,V,D,skew", [
    (1, 1, 1, 1, 0), (1, 1, 5, 64, 0), (7, 3, 4, 33, 0), (40, 5, 1000, 129, 0), (300, 4, 17, 100, 0),
    (128, 9, 513, 260, 1), (64, 2, 1, 768, 0), (1025, 1, 70000, 8, 1), (2111, 8, 97, 64, 1),
    (2111, 8, 40000, 20, 1)])
def test_embed_bwd(T, B, V, D, skew, dt):
    rng = np.random.default_rng(T + V)
    n = rng.integers(-1, V + 1, (T, B))
    if skew:  # half of all ids the same one
        n[rng.random((T, B)) < 0.5] = V // 3
    dx = _rand(rng, (T, B, D), dt)
    ids = torch.from_numpy(n).cuda()
    out = torch.full((V, D), float("nan"), device="cuda")
    g.embed_bwd(ids, dx, V, 0.3, out=out)
    ref = lm_ref.embed_grad(n, _np(dx), V, np.float32(0.3))
    mag = lm_ref.embed_grad(n, np.abs(_np(dx)), V, np.float32(0.3))
    cnt = np.bincount(n[(n >= 0) & (n < V)], minlength=V)[:, None]
    _within("dtable", out, ref, (cnt + 2) * U * mag)
    # the order of the sums is the ids' alone
    again = g.embed_bwd(ids.int(), dx, V, 0.3)
    assert torch.equal(out, again)
    # batch-first ids read time-first
    assert torch.equal(out, g.embed_bwd(ids.t().contiguous().t(), dx, V, 0.3))


@pytest.mark.parametrize("M,V,D", [(70001, 1000, 8), (300007, 50000, 4), (300007, 3, 5), (5000, 300000, 4),
                                   (1000, 600000, 1)])
def test_embed_bwd_many_ids(M, V, D):
    """The blocked sort's larger blocks and its third pass, against sums in
    64 bits on the device."""
    gen = torch.Generator(device="cuda").manual_seed(M)
    ids = torch.randint(-1, V + 1, (M,), generator=gen, device="cuda")
    ids[::3] = V // 2
    dx = torch.randn((M, D), generator=gen, device="cuda")
    out = g.embed_bwd(ids, dx, V, 0.5)
    ok = (ids >= 0) & (ids < V)
    ref, mag = (torch.zeros((V, D), dtype=torch.float64, device="cuda").index_add_(
        0, ids[ok], t[ok].double() * 0.5) for t in (dx, dx.abs()))
    cnt = torch.bincount(ids[ok], minlength=V)[:, None]
    assert ((out - ref).abs() <= (cnt + 2) * U * mag).all()
    assert torch.equal(out, g.embed_bwd(ids, dx, V, 0.5))


def test_embed_bwd_all_padding():
    out = torch.full((11, 5), float("nan"), device="cuda")
    g.embed_bwd(torch.full((3, 4), -1, device="cuda"), torch.ones((3, 4, 5), device="cuda"), 11,
                out=out)
    assert not out.any()


def test_embed_bwd_is_the_adjoint():
    """<dE, F> = <dx, embed(F)>: the lookup is linear in the table."""
    rng = np.random.default_rng(9)
    ids = torch.from_numpy(rng.integers(0, 50, (37, 3))).cuda()
    dx, F = _rand(rng, (37, 3, 65), "f32"), _rand(rng, (50, 65), "f32")
    a = (g.embed_bwd(ids, dx, 50, 1.5).double() * F.double()).sum().item()
    b = (dx.double() * g.embed_fwd(ids, F, 1.5).double()).sum().item()
    assert abs(a - b) <= 1e-5 * (dx.double().abs() * 1.5).sum().item()


# ------------------------------------------------- token log probabilities
def _logits(rng, M, V, dt, kind):
    x = rng.standard_normal((M, V)).astype(np.float32) * 3
    if kind == "banned":
        x[rng.random((M, V)) < 0.6] = -np.inf
        x[0] = -np.inf                      # nothing allowed
        if M > 1:
            x[1] = -np.inf
            x[1, V // 2] = 1.5              # one entry allowed
    elif kind == "ties":
        x = np.round(x)
    elif kind == "equal":
        x[:] = 0.25
    elif kind == "sorted":
        x = np.sort(x, axis=1)
    elif kind == "lowest":
        x[rng.random((M, V)) < 0.5] = np.finfo(np.float32).min if dt == "f32" else -3.38953139e38
    elif kind == "zeros":
        x = np.where(rng.random((M, V)) < 0.5, -0.0, 0.0).astype(np.float32)
    return torch.from_numpy(x).to(DT[dt]).cuda()


def _check_logprobs(x, tok, K, **kw):
    r = g.token_logprobs(x, tok, top=K, **kw)
    ref = lm_ref.logprobs(_np(x), tok.cpu().numpy(), K)
    for k in ("logp", "lse"):
        fin = np.where(np.isfinite(ref[k]), np.abs(ref[k]), 0)
        _within(k, r[k], ref[k], 2e-5 + 2 * U * fin)
    _within("entropy", r["entropy"], ref["entropy"], 2e-4)
    if K:
        assert np.array_equal(r["top_id"].cpu().numpy(), ref["top_id"])
        fin = np.where(np.isfinite(ref["top_logp"]), np.abs(ref["top_logp"]), 0)
        _within("top_logp", r["top_logp"], ref["top_logp"], 2e-5 + 2 * U * fin)
    return r


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["plain", "banned", "ties", "equal", "sorted", "lowest", "zeros"])
@pytest.mark.parametrize("M,V,K", [(1, 1, 1), (3, 2, 2), (4, 65, 20), (5, 1000, 64), (3, 8193, 8),
                                   (2, 8192, 0), (3, 20011, 33)])
def test_token_logprobs(M, V, K, kind, dt):
    rng = np.random.default_rng(V + K)
    x = _logits(rng, M, V, dt, kind)
    tok = torch.from_numpy(rng.integers(0, V, M)).cuda()
    if M > 2:
        tok[2] = -1
    _check_logprobs(x, tok, K)
    r = _check_logprobs(x, tok.int(), K)
    assert r["logp"].dtype == torch.float32


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_token_logprobs_row_strides(dt):
    """Rows that start anywhere in their 16 bytes, a padded vocabulary, [T,B,V]."""
    rng = np.random.default_rng(5)
    big = _logits(rng, 6, 9000, dt, "plain")
    tok = torch.from_numpy(rng.integers(0, 700, 6)).cuda()
    for lo, hi in ((0, 777), (1, 778), (3, 1500), (7, 8999), (5, 712)):
        _check_logprobs(big[:, lo:hi], tok, 5)
    x = big[:, :800].contiguous().view(2, 3, 800)
    r = g.token_logprobs(x, tok.view(2, 3), top=4)
    s = g.token_logprobs(x.view(6, 800), tok, top=4)
    assert tuple(r["top_id"].shape) == (2, 3, 4)
    for k in s:
        assert torch.equal(r[k].reshape(s[k].shape), s[k]), k


def test_token_logprobs_not_finite():
    x = torch.zeros((4, 9001), device="cuda")
    x[0, 17] = float("nan")
    x[1, 8888] = float("inf")
    x[2, 3:] = float("nan")
    tok = torch.tensor([1, 2, 0, 4], device="cuda")
    r = g.token_logprobs(x, tok, top=3)
    for k in ("logp", "entropy", "lse"):
        assert torch.isnan(r[k][:3]).all() and torch.isfinite(r[k][3]).all(), k
    ids = r["top_id"].cpu()
    assert ids[0].tolist() == [17, 0, 1] and ids[1].tolist() == [8888, 0, 1]
    assert ids[2].tolist() == [3, 4, 5] and ids[3].tolist() == [0, 1, 2]


def test_token_logprobs_offsets_past_32_bits():
    M, V = 60000, 40001  # 2.4e9 logits
    x = torch.zeros((M, V), dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([0, 53686, 53688, M - 1], device="cuda")
    rng = np.random.default_rng(2)
    x[rows] = _rand(rng, (4, V), "bf16", 3.0)
    tok = torch.full((M,), 40000, device="cuda")
    r = g.token_logprobs(x, tok, top=3)
    want = g.token_logprobs(x[rows], tok[rows], top=3)
    assert torch.equal(r["top_id"][rows], want["top_id"])
    for k in ("logp", "lse", "top_logp", "entropy"):  # rows start elsewhere: other partial sums
        assert (r[k][rows] - want[k]).abs().max() <= (2e-4 if k == "entropy" else 2e-5), k
    assert abs(r["lse"][1].item() - np.log(V)) < 1e-5
    dlogp = torch.ones((M,), device="cuda")
    g.token_logprobs_bwd(x, tok, r["lse"], r["entropy"], dlogp, out=x)  # in place
    assert abs(x[M - 2, 40000].item() - 1) < 1e-2 and abs(x[M - 2, :-1].double().sum().item() + 1) < 2e-2


def _grad_bound(x, lse, H, dlogp, dent, dt, ref):
    with np.errstate(invalid="ignore"):
        lp = np.where(np.isfinite(x), x - lse[:, None], -200.0)
    lp = np.where(np.isfinite(lp), lp, -200.0)
    p = np.exp(lp)
    l1 = np.where(np.isfinite(lse), np.abs(lse), 0)[:, None]
    rel = U * (4 * l1 + 4 * np.abs(lp) + 16)
    mag = p * (np.abs(dlogp)[:, None] + np.abs(dent)[:, None] * (np.abs(lp) + np.abs(H)[:, None] + 1))
    # the entropy given back is float32, and 2e-4 off at most
    return mag * rel + p * np.abs(dent)[:, None] * 2e-4 + _r(ref, dt) + 4 * U * np.abs(ref) + 1e-30


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["plain", "banned", "lowest"])
@pytest.mark.parametrize("M,V", [(1, 1), (3, 7), (4, 1000), (3, 4097), (5, 10001)])
def test_token_logprobs_bwd(M, V, kind, dt):
    rng = np.random.default_rng(M * V)
    x = _logits(rng, M, V, dt, kind)
    n = rng.integers(0, V, M)
    if M > 2:
        n[2] = V  # no token
    tok = torch.from_numpy(n).cuda()
    dl, de = _rand(rng, (M,), "f32"), _rand(rng, (M,), "f32")
    f = g.token_logprobs(x, tok)
    xs, lse, H = _np(x), _np(f["lse"]), _np(f["entropy"])
    zero = np.zeros(M)
    for a, b in ((dl, de), (dl, None), (None, de), (None, None)):
        an, bn = (zero if t is None else _np(t) for t in (a, b))
        ref = lm_ref.logprobs_grad(xs, n, an, bn)
        d = g.token_logprobs_bwd(x, tok, f["lse"], f["entropy"], a, b)
        assert d.dtype == x.dtype
        _within("dlogits", d, ref, _grad_bound(xs, lse, H, an, bn, dt, ref))
    y = x.clone()
    assert g.token_logprobs_bwd(y, tok, f["lse"], f["entropy"], dl, de, out=y) is y
    assert torch.equal(y, g.token_logprobs_bwd(x, tok, f["lse"], f["entropy"], dl, de))


def test_token_logprobs_bwd_row_strides():
    rng = np.random.default_rng(8)
    big, other = _logits(rng, 5, 3000, "f32", "plain"), torch.zeros((5, 3007), device="cuda")
    tok = torch.from_numpy(rng.integers(0, 500, 5)).cuda()
    dl, de = _rand(rng, (5,), "f32"), _rand(rng, (5,), "f32")
    for lo, hi, at in ((0, 800, 0), (1, 1500, 1), (3, 2999, 2), (2, 600, 7)):
        x, o = big[:, lo:hi], other[:, at:at + hi - lo]
        other.zero_()
        f = g.token_logprobs(x, tok)
        g.token_logprobs_bwd(x, tok, f["lse"], f["entropy"], dl, de, out=o)
        want = g.token_logprobs_bwd(x.contiguous(), tok, f["lse"], f["entropy"], dl, de)
        assert torch.equal(o, want)
        assert not other[:, :at].any() and not other[:, at + hi - lo:].any()


def test_token_logprobs_gradient_by_differences():
    """Central differences of the 64-bit definition at the library's gradient."""
    rng = np.random.default_rng(4)
    x = _logits(rng, 3, 50, "f32", "plain")
    tok = torch.tensor([3, 0, 49], device="cuda")
    dl, de = _rand(rng, (3,), "f32"), _rand(rng, (3,), "f32")
    f = g.token_logprobs(x, tok)
    d = _np(g.token_logprobs_bwd(x, tok, f["lse"], f["entropy"], dl, de))

    def loss(y):
        r = lm_ref.logprobs(y, tok.cpu().numpy(), 1)
        return (r["logp"] * _np(dl)).sum() + (r["entropy"] * _np(de)).sum()
    xs, h = _np(x), 1e-5
    for _ in range(20):
        v = rng.standard_normal(xs.shape)
        num = (loss(xs + h * v) - loss(xs - h * v)) / (2 * h)
        # h^2 of the third derivative, rounding 1e-16 * 50 / h, float32 gradient
        assert abs(num - (d * v).sum()) <= 1e-5 * np.abs(d * v).sum() + 1e-8


# -------------------------------------------------------- linear attention
def _lin_case(seed, T, B, NH, NKV, Dk, Dv, dt, layout="dense", decay="mixed"):
    rng = np.random.default_rng(seed)
    widths = [NH * Dk, NKV * Dk, NKV * Dv]
    if layout == "fused":       # slices of one projection
        x = _rand(rng, (T, B, sum(widths)), dt)
        parts = x.split(widths, -1)
    elif layout == "bt":        # batch-first arrays read time-first
        parts = [_rand(rng, (B, T, w), dt).transpose(0, 1) for w in widths]
    elif layout == "odd":       # rows that start at an odd element
        parts = [_rand(rng, (T, B, w + 3), dt)[..., 1:w + 1] for w in widths]
    else:
        parts = [_rand(rng, (T, B, w), dt) for w in widths]
    q, k, v = (p.unflatten(-1, (n, -1)) for p, n in zip(parts, (NH, NKV, NKV)))
    if decay == "none":
        ld = np.zeros(NH)
    elif decay == "all":
        ld = np.full(NH, -np.inf)
    else:
        ld = -np.exp(rng.uniform(np.log(1e-3), np.log(4.0), NH))
        if NH > 2:
            ld[1], ld[2] = 0.0, -np.inf
    gd = torch.from_numpy(ld.astype(np.float32)).cuda()
    S0 = _rand(rng, (B, NH, Dk, Dv), "f32")
    return rng, q, k, v, gd, S0


def _c(T, Dk, dt):
    return (Dk + T + 64) * U + 3e-6 + (3 * 2.0 ** -17 if dt == "bf16" else 0.0)


def _check_lin(T, B, NH, NKV, Dk, Dv, dt, layout="dense", decay="mixed", with_state=True, seed=0):
    rng, q, k, v, gd, S0 = _lin_case(seed + T + Dk, T, B, NH, NKV, Dk, Dv, dt, layout, decay)
    S0 = S0 if with_state else None
    sc = 0.37
    o, S = g.linattn_fwd(q, k, v, gd, S0, scale=sc)
    assert o.dtype == q.dtype and S.dtype == torch.float32
    n = [_np(t) for t in (q, k, v, gd)]
    s0 = None if S0 is None else _np(S0)
    ro, rS = lm_ref.linattn(*n, s0, sc)
    mo, mS = lm_ref.linattn(*[np.abs(t) for t in n[:3]], n[3], None if s0 is None else np.abs(s0), sc)
    c = _c(T, max(Dk, Dv), dt)
    _within("o", o, ro, c * mo + _r(ro, dt))
    _within("S", S, rS, c * mS)
    do = _rand(rng, (T, B, NH, Dv), dt)
    dST = _rand(rng, (B, NH, Dk, Dv), "f32") if with_state else None
    r = g.linattn_bwd(q, k, v, gd, do, S0, dST, scale=sc)
    dn, dS = _np(do), None if dST is None else _np(dST)
    ref = lm_ref.linattn_grad(*n, s0, dn, dS, sc)
    mag = lm_ref.linattn_grad(*[np.abs(t) for t in n[:3]], n[3], None if s0 is None else np.abs(s0),
                              np.abs(dn), None if dS is None else np.abs(dS), sc)
    for name in ("dq", "dk", "dv", "dS0"):
        _within(name, r[name], ref[name],
                c * mag[name] + _r(ref[name], dt if name != "dS0" else "f32"))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,B,NH,NKV,Dk,Dv", [
    (1, 1, 1, 1, 1, 1), (2, 1, 1, 1, 16, 16), (5, 2, 3, 1, 7, 9), (31, 1, 2, 2, 32, 32),
    (32, 2, 2, 1, 64, 64), (33, 1, 3, 3, 48, 80), (64, 1, 2, 2, 128, 128), (65, 2, 4, 2, 96, 64),
    (127, 1, 2, 1, 33, 130), (129, 1, 1, 1, 256, 192), (200, 1, 2, 2, 100, 256),
    (300, 2, 3, 3, 64, 128), (1000, 1, 1, 1, 40, 24)])
def test_linattn(T, B, NH, NKV, Dk, Dv, dt):
    _check_lin(T, B, NH, NKV, Dk, Dv, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["fused", "bt", "odd"])
def test_linattn_layouts(layout, dt):
    _check_lin(70, 3, 4, 2, 64, 64, dt, layout)
    _check_lin(70, 3, 2, 2, 36, 20, dt, layout)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("decay", ["none", "all"])
def test_linattn_decays(decay, dt):
    _check_lin(150, 2, 3, 3, 64, 32, dt, decay=decay)
    _check_lin(90, 1, 2, 1, 64, 64, dt, decay=decay, with_state=False)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_linattn_without_state(dt):
    _check_lin(333, 1, 2, 2, 64, 64, dt, with_state=False)
    _check_lin(1, 2, 2, 2, 64, 64, dt, with_state=False)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,NH,NKV,Dk,Dv", [(1, 1, 1, 1, 1), (3, 2, 1, 64, 64), (2, 3, 3, 100, 36),
                                            (1, 2, 2, 256, 256), (5, 4, 2, 33, 77)])
def test_linattn_step(B, NH, NKV, Dk, Dv, dt):
    """Token by token equals the definition; in place and to another state."""
    T = 6
    _, q, k, v, gd, S0 = _lin_case(B + Dk, T, B, NH, NKV, Dk, Dv, dt, "fused")
    n = [_np(t) for t in (q, k, v, gd)]
    ro, rS = lm_ref.linattn(*n, _np(S0), 0.2)
    mo, mS = lm_ref.linattn(*[np.abs(t) for t in n[:3]], n[3], np.abs(_np(S0)), 0.2)
    keep, S, os = S0.clone(), S0, []
    for t in range(T):
        S_out = torch.empty_like(S) if t == 0 else None
        o, S2 = g.linattn_step(q[t:t + 1], k[t:t + 1], v[t:t + 1], gd, S, scale=0.2, S_out=S_out)
        assert (S2 is S) == (t > 0)
        S = S2
        os.append(o)
    assert torch.equal(S0, keep)
    c = _c(T, Dk, "f32")
    _within("o", torch.cat(os), ro, c * mo + _r(ro, dt))
    _within("S", S, rS, c * mS)


def test_linattn_prompt_then_steps_and_state_in_place():
    _, q, k, v, gd, S0 = _lin_case(1, 100, 2, 2, 2, 64, 64, "f32")
    o, S = g.linattn_fwd(q, k, v, gd, S0, scale=0.1)
    S1 = S0.clone()
    o1, S2 = g.linattn_fwd(q[:77], k[:77], v[:77], gd, S1, scale=0.1, out={"S": S1})
    assert S2 is S1
    outs = [o1]
    for t in range(77, 100):
        outs.append(g.linattn_step(q[t:t + 1], k[t:t + 1], v[t:t + 1], gd, S1, scale=0.1)[0])
    assert (torch.cat(outs) - o).norm() <= 1e-5 * o.norm()
    assert (S1 - S).norm() <= 1e-5 * S.norm()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,B,NH,Dk,Dv", [(200, 1, 2, 64, 64), (1100, 1, 2, 64, 48), (1500, 2, 3, 128, 128),
                                          (700, 1, 1, 33, 70)])
def test_linattn_state_in_place_over_segments(T, B, NH, Dk, Dv, dt):
    """The final state over the initial one, where the sequence runs in
    segments at once: the same bits as into another tensor."""
    _, q, k, v, gd, S0 = _lin_case(T, T, B, NH, NH, Dk, Dv, dt)
    assert g.workspace_size_linattn(g.OP_LIN_FWD, g.LinDims(T, B, NH, NH, Dk, Dv),
                                    g.RNN_BF16 if dt == "bf16" else g.RNN_F32) > 0
    o, S = g.linattn_fwd(q, k, v, gd, S0)
    for _ in range(3):
        S1 = S0.clone()
        o1, S2 = g.linattn_fwd(q, k, v, gd, S1, out={"S": S1})
        assert S2 is S1 and torch.equal(S1, S) and torch.equal(o1, o)


def test_linattn_strides_past_32_bits():
    _, q, k, v, gd, S0 = _lin_case(6, 3, 1, 2, 2, 32, 32, "bf16")
    far = torch.empty((3, 1, 1 << 30, 1), dtype=torch.bfloat16, device="cuda")
    fq = far[:, :, 64:128].view(3, 1, 2, 32)
    fq.copy_(q)
    o, S = g.linattn_fwd(fq, k, v, gd, S0)
    w, S1 = g.linattn_fwd(q, k, v, gd, S0)
    assert torch.equal(o, w) and torch.equal(S, S1)


def test_linattn_keys_shared_by_the_batch():
    """Keys and values broadcast over the batch (stride 0): their gradients
    are those of a copy for each row, which sum to the shared one's."""
    _, q, k, v, gd, S0 = _lin_case(2, 50, 3, 2, 2, 32, 32, "f32")
    k1, v1 = k[:, :1].expand(-1, 3, -1, -1), v[:, :1].expand(-1, 3, -1, -1)
    do = torch.randn_like(q)
    a = g.linattn_bwd(q, k1, v1, gd, do, S0)
    b = g.linattn_bwd(q, k1.contiguous(), v1.contiguous(), gd, do, S0)
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_linattn_gradient_by_differences():
    """The loss is linear in each of q, k (v fixed), v, S0: a difference of
    any size is exact up to rounding."""
    rng, q, k, v, gd, S0 = _lin_case(11, 90, 2, 4, 2, 32, 48, "f32")
    do, dST = _rand(rng, (90, 2, 4, 48), "f32"), _rand(rng, tuple(S0.shape), "f32")
    r = g.linattn_bwd(q, k, v, gd, do, S0, dST, scale=0.3)

    def loss(q, k, v, S0):
        o, S = g.linattn_fwd(q, k, v, gd, S0, scale=0.3)
        return ((o.double() * do.double()).sum() + (S.double() * dST.double()).sum()).item()
    args = {"q": q, "k": k, "v": v, "S0": S0}
    for name, t in args.items():
        d = torch.randn_like(t)
        num = (loss(**{**args, name: t + d}) - loss(**{**args, name: t - d})) / 2
        grad = r["d" + name].double() * d.double()
        # rounding of the two losses: 1e-6 of the sum of magnitudes, far below sqrt(n) of it
        assert abs(num - grad.sum().item()) <= 1e-3 * grad.norm().item() + 1e-4 * abs(num), name


# ------------------------------------------------------------------ streams
def test_another_stream():
    """Calls and their workspaces on a stream of their own, with work before
    and after them on the current one."""
    rng = np.random.default_rng(1)
    side = torch.cuda.Stream()
    ids = torch.from_numpy(rng.integers(0, 500, (64, 4))).cuda()
    dx = _rand(rng, (64, 4, 64), "f32")
    x = _rand(rng, (8, 20000), "f32", 3.0)
    tok = torch.from_numpy(rng.integers(0, 20000, 8)).cuda()
    _, q, k, v, gd, S0 = _lin_case(3, 300, 1, 2, 2, 64, 64, "bf16")
    want = (g.embed_bwd(ids, dx, 500), g.token_logprobs(x, tok, top=5)["top_logp"],
            g.linattn_fwd(q, k, v, gd, S0)[0])
    torch.cuda.synchronize()
    for _ in range(5):
        side.wait_stream(torch.cuda.current_stream())
        got = (g.embed_bwd(ids, dx, 500, stream=side),
               g.token_logprobs(x, tok, top=5, stream=side)["top_logp"],
               g.linattn_fwd(q, k, v, gd, S0, stream=side)[0])
        torch.full((1 << 20,), 7.0, device="cuda")  # reuses what the current stream frees
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_captured_in_a_graph():
    """Calls with their outputs and workspaces given, captured and replayed
    over changing inputs with eager work between the replays."""
    rng = np.random.default_rng(12)
    ids = torch.from_numpy(rng.integers(-1, 3000, (600, 9))).cuda()
    dx = _rand(rng, (600, 9, 64), "f32")
    x, tok = _rand(rng, (6, 20001), "bf16", 3.0), torch.from_numpy(rng.integers(0, 20001, 6)).cuda()
    _, q, k, v, gd, S0 = _lin_case(4, 900, 1, 2, 1, 64, 64, "bf16")
    do = _rand(rng, (900, 1, 2, 64), "bf16")
    u8 = lambda n: torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")  # noqa: E731
    d = g.LinDims(900, 1, 2, 1, 64, 64)
    w = [u8(g.workspace_size_embed_bwd(600, 9, 3000, 64)), u8(g.workspace_size_logprobs(6, 20001, 7)),
         u8(g.workspace_size_linattn(g.OP_LIN_FWD, d, 1)), u8(g.workspace_size_linattn(g.OP_LIN_BWD, d, 1))]

    def calls():
        r = g.token_logprobs(x, tok, top=7, ws=w[1])
        b = g.linattn_bwd(q, k, v, gd, do, S0, ws=w[3])
        return [g.embed_bwd(ids, dx, 3000, ws=w[0]), *r.values(),
                *g.linattn_fwd(q, k, v, gd, S0, ws=w[2]), *b.values()]
    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = calls()
    for i in range(4):
        dx.mul_(1.0 + i)
        ids.copy_(ids.roll(i, 0))
        x.copy_(x.roll(i, 1))
        q.copy_(q.flip(0))
        graph.replay()
        got = [t.clone() for t in out]
        for a, b in zip(got, calls()):
            assert torch.equal(a, b), i
        torch.cuda.synchronize()
