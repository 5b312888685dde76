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
