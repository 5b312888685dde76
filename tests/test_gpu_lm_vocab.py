"""Token log probabilities over the longest vocabularies: more chunks than a
wave has lanes (V > 524288), the join's largest shared memory (V = 1000000 with
64 alternatives), and more candidates at the join's bound than it keeps."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gru_recurrence_amd as g  # noqa: E402

U = 2.0 ** -24
CHUNK = 8192  # logits that one workgroup holds
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _reference(x, tok, K):
    x = x.double().cpu().numpy()
    m = x.max(1, keepdims=True)
    lse = (m + np.log(np.exp(x - m).sum(1, keepdims=True)))[:, 0]
    lp = x - lse[:, None]
    p = np.exp(lp)
    ent = -(p * np.where(p > 0, lp, 0.0)).sum(1)
    ids = np.argsort(-x, 1, kind="stable")[:, :K]  # ties to the lowest index
    rows = np.arange(len(x))
    return dict(lse=lse, entropy=ent, logp=lp[rows, tok], top_id=ids, top_logp=lp[rows[:, None], ids])


def _check(x, K, tok):
    r = {k: v.double().cpu().numpy()
         for k, v in g.token_logprobs(x, torch.from_numpy(tok).cuda(), top=K).items()}
    ref = _reference(x, tok, K)
    for k in ref:
        if k == "top_id":
            if K:
                assert np.array_equal(r[k], ref[k]), k
        elif K or k != "top_logp":
            # e^z and sums of a row in float32, |l| and |lse| below 40: 2e-5; the
            # entropy's terms are |z| times those of the sum: 2e-4
            fin = np.isfinite(ref[k])
            assert np.array_equal(r[k][~fin], ref[k][~fin]), k
            bound = 2e-4 if k == "entropy" else 2e-5 + 2 * U * np.abs(ref[k][fin])
            assert (np.abs(r[k][fin] - ref[k][fin]) <= bound).all(), k


def _logits(rng, M, V, kind):
    x = rng.standard_normal((M, V)).astype(np.float32) * 3
    late = 64 * CHUNK
    if kind == "late":       # what counts lies in chunks past the 64th
        x[:, late + rng.integers(0, V - late, 70)] += 20.0
    elif kind == "masked":   # nothing but a few entries past the 64th chunk, ruled out chunks before
        y = np.full_like(x, -np.inf)
        at = rng.permutation(V - late)[:100] + late
        y[:, at] = x[:, at]
        x = y
    elif kind == "ties":
        x = np.round(x)
    elif kind == "crowded":  # each chunk's own top fills all but one of the alternatives
        x[:] = 0.0
        for c in range(0, V, CHUNK):
            n = min(63, V - c)
            x[:, c + rng.permutation(min(CHUNK, V - c))[:n]] = 1.0 + rng.random(n).astype(np.float32)
    return x


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["plain", "late", "masked", "ties", "crowded"])
@pytest.mark.parametrize("V,K", [(524289, 3), (600001, 20), (1000000, 64), (1000000, 0)])
def test_long_vocabularies(V, K, kind, dt):
    rng = np.random.default_rng(V + K)
    x = torch.from_numpy(_logits(rng, 2, V, kind)).to(DT[dt]).cuda()
    _check(x, K, np.array([V - 1, 64 * CHUNK]))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V", [150000, 200000, 400001])
def test_more_candidates_than_the_join_keeps(V, dt):
    """63 of each chunk's entries lie above every chunk's 64th: over 1024 keys
    reach the join's bound."""
    assert 63 * (V // CHUNK) > 1024
    x = torch.from_numpy(_logits(np.random.default_rng(V), 3, V, "crowded")).to(DT[dt]).cuda()
    _check(x, 64, np.array([0, V // 2, V - 1]))
