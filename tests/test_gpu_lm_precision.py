"""What linear attention keeps: values whose every bit has to survive, states
and decays, and a decay that is not a number."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gru_recurrence_amd as g  # noqa: E402

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
TYPES = pytest.mark.parametrize("dt", ["bf16", "f32"])


def _dev(a, dt):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(DT[dt]).cuda()


def _bf(x, dt):
    return torch.from_numpy(x.astype(np.float32)).to(DT[dt]).double().numpy()


@TYPES
@pytest.mark.parametrize("T", [1, 5, 200, 2500])
def test_linattn_decay_that_is_not_a_number(T, dt):
    """A NaN decay shows in its own head and no other, whichever form runs."""
    rng = np.random.default_rng(T)
    q, k, v, do = (_dev(rng.standard_normal((T, 2, 3, 32)), dt) for _ in range(4))
    gd = torch.tensor([-0.1, float("nan"), -float("inf")], device="cuda")
    S0 = _dev(rng.standard_normal((2, 3, 32, 32)), "f32")
    o, S = g.linattn_fwd(q, k, v, gd, S0)
    r = g.linattn_bwd(q, k, v, gd, do, S0, S0)
    # the last token's dk and dv take no decay but through X, which is NaN all the same
    for name, t, axis in (("o", o, 2), ("S", S, 1), *((n, r[n], 2) for n in ("dq", "dk", "dv")),
                          ("dS0", r["dS0"], 1)):
        bad = torch.isnan(t)
        assert bad.select(axis, 1).all(), name
        assert not bad.select(axis, 0).any() and not bad.select(axis, 2).any(), name


@TYPES
@pytest.mark.parametrize("T", [2, 40, 200, 1500])
def test_linattn_states_are_float32(T, dt):
    """One token's k^T v, decayed over the rest of the sequence, is a single
    term: off by u = 2^-24 for each of at most ten roundings, three for each
    chunk of 32 rows or more that it is carried over, and 2.1 for each unit of
    the exponent n log2 a (the decay's logarithm and its multiples, ln 2 of
    their error, and a hardware exponential)."""
    rng = np.random.default_rng(T)
    D, NH = 64, 4
    ld = (-np.array([0.5, 3.0, 8.0, 20.0]) / T).astype(np.float32)
    k, v = rng.standard_normal((2, 1, 2, NH, D))
    rest = np.zeros((T - 1, 2, NH, D))
    first, last = (_dev(np.concatenate(p), dt) for p in ((k, rest), (rest, k)))
    firstv, lastv = (_dev(np.concatenate(p), dt) for p in ((v, rest), (rest, v)))
    gd, zero = torch.from_numpy(ld).cuda(), torch.zeros_like(first)
    kv = _bf(k[0], dt)[..., :, None] * _bf(v[0], dt)[..., None, :]
    n = ld.astype(np.float64)[None, :, None, None]

    def near(name, t, steps):
        want = kv * np.exp(n * steps)
        c = (2.1 * np.abs(n) * T * 1.4427 + 3 * (T / 32 + 1) + 10) * U
        err = np.abs(t.double().cpu().numpy() - want)
        assert (err <= c * np.abs(want)).all(), (name, float((err / (c * np.abs(want) + 1e-300)).max()))
    near("S", g.linattn_fwd(zero, first, firstv, gd)[1], T - 1)
    near("dS0", g.linattn_bwd(last, zero, zero, gd, lastv, scale=1.0)["dS0"], T)


def _pairs(rng, n, D):
    """n rows of whole numbers up to 255 in neighbours that differ in one place
    by one: products with any row are large, their differences small."""
    x = rng.integers(-255, 256, (n, D))
    x[1::2] = x[0::2]
    x[1::2, rng.integers(0, D)] += 1
    return np.clip(x, -256, 255)


def _differences(n, D):
    """Column c takes row 2c less row 2c + 1."""
    z = np.zeros((n, D), np.int64)
    for c in range(min(D, n // 2)):
        z[2 * c, c], z[2 * c + 1, c] = 1, -1
    return z


@TYPES
@pytest.mark.parametrize("T,D", [(40, 16), (64, 32), (64, 128), (150, 64)])
def test_linattn_products_of_rows_keep_every_bit(T, D, dt):
    """Without decay and with whole numbers every product and sum is exact in
    float32, so the outputs are the exact ones, rounded once: x . y reaches 2^23
    and its odd last bits are all that is left of z's differences."""
    rng = np.random.default_rng(T + D)
    x, y, z = rng.integers(-255, 256, (T, D)), _pairs(rng, T, D), _differences(T, D)
    low = np.tril(np.ones((T, T), np.int64))
    want = _bf(((x @ y.T) * low) @ z, dt)                         # row i: sum over j <= i
    assert np.abs((x @ y.T)).max() < 2 ** 24
    rev = lambda t: t[::-1]  # noqa: E731
    X, Y, Z = (_dev(t.reshape(T, 1, 1, D), dt) for t in (x, y, z))
    Xr, Yr, Zr = (_dev(rev(t).reshape(T, 1, 1, D), dt) for t in (x, y, z))
    gd = torch.zeros(1, device="cuda")
    o, _ = g.linattn_fwd(X, Y, Z, gd, scale=1.0)
    got = {"o": o, "dq": g.linattn_bwd(Y, Z, Y, gd, X, scale=1.0)["dq"],   # x, y, z = do, v, k
           "dk": g.linattn_bwd(Zr, Zr, Xr, gd, Yr, scale=1.0)["dk"].flip(0),  # v, do, q
           "dv": g.linattn_bwd(Yr, Xr, Yr, gd, Zr, scale=1.0)["dv"].flip(0)}  # k, q, do
    for name, t in got.items():
        assert np.array_equal(t.double().cpu().numpy()[:, 0, 0], want), name


@TYPES
@pytest.mark.parametrize("T,D", [(3, 16), (70, 64), (64, 128), (1500, 128)])
def test_linattn_outputs_see_every_bit_of_the_state(T, D, dt):
    """The state's share of an output is the difference of two of its rows, of
    24 bits each."""
    rng = np.random.default_rng(T * D)
    S = rng.integers(2 ** 22, 2 ** 23, (D, D))
    S[1::2] = S[0::2] - rng.integers(-255, 256, (D // 2, D))
    x = np.zeros((T, D), np.int64)
    m = rng.integers(0, D // 2, T)
    x[np.arange(T), 2 * m], x[np.arange(T), 2 * m + 1] = 1, -1
    want = (x @ S).astype(np.float64)                             # at most 255: exact in bf16
    z = torch.zeros((T, 1, 1, D), dtype=DT[dt], device="cuda")
    X, gd = _dev(x.reshape(T, 1, 1, D), dt), torch.zeros(1, device="cuda")
    St, Sr = _dev(S.reshape(1, 1, D, D), "f32"), _dev(S.T.reshape(1, 1, D, D), "f32")
    o, ST = g.linattn_fwd(X, z, z, gd, St, scale=1.0)
    got = {"o": o, "dq": g.linattn_bwd(z, z, z, gd, X, Sr, scale=1.0)["dq"],
           "dk": g.linattn_bwd(z, z, X, gd, z, None, Sr, scale=1.0)["dk"],
           "dv": g.linattn_bwd(z, X, z, gd, z, None, St, scale=1.0)["dv"]}
    for name, t in got.items():
        assert np.array_equal(t.double().cpu().numpy()[:, 0, 0], want), name
    assert torch.equal(ST, St)
