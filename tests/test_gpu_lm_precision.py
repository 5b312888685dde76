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
