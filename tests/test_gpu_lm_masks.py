"""Alternatives of rows that a mask rules out in part or in whole, and of rows
with many equal entries: which ones they are, and that they cost no cliff."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gru_recurrence_amd as g  # noqa: E402

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
LOWEST = {"bf16": -3.3895313892515355e38, "f32": float(np.finfo(np.float32).min)}


def _rows(kind, V, dt, rng):
    x = rng.standard_normal((6, V)).astype(np.float32) * 3
    mask = LOWEST[dt] if kind.endswith("lowest") else -np.inf
    if kind.startswith("block"):     # reserved ids: all of some chunks
        x[:, 5000:min(V - 3, 21000)] = mask
    elif kind.startswith("allowed"):  # few allowed entries, 0 to 5 of them a chunk
        y = np.full_like(x, mask)
        for r, n in enumerate((1, 2, 3, 5, 9, 40)):
            at = rng.permutation(V)[:n]
            y[r, at] = x[r, at]
        x = y
    elif kind == "steps":            # ties at the bound among smaller entries, few above
        x = np.where(rng.random((6, V)) < 0.4, 1.0, np.minimum(x, 0.5)).astype(np.float32)
        x[:, rng.permutation(V)[:7]] = 4.0
    elif kind == "late ties":        # ties at the bound only towards the end
        x[:] = -1.0 - rng.random((6, V)).astype(np.float32)
        x[:, V // 2:] = 2.0
    elif kind == "columns":          # over a thousand entries above every bound
        x[:] = -np.abs(x)
        x[:, np.arange(V) % 128 < 17] += 50.0
    elif kind == "not a number":
        x[:, :V // 2] = np.nan
        x[:, V // 2:] = np.inf
    return torch.from_numpy(x).to(DT[dt])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["block", "block lowest", "allowed", "allowed lowest", "steps",
                                  "late ties", "columns", "not a number"])
@pytest.mark.parametrize("V,K", [(7000, 20), (8192, 64), (40003, 5), (40003, 33), (40003, 64)])
def test_alternatives(V, K, kind, dt):
    """Largest first, ties to the lowest index, NaN above everything: all exact."""
    x = _rows(kind, V, dt, np.random.default_rng(V + K))
    r = g.token_logprobs(x.cuda(), torch.zeros(6, dtype=torch.int64, device="cuda"), top=K)
    y = x.double().numpy()
    key = np.where(np.isnan(y), np.inf, y)
    order = np.stack([np.lexsort((np.arange(V), -key[i], ~np.isnan(y[i]))) for i in range(6)])
    assert np.array_equal(r["top_id"].cpu().numpy(), order[:, :K])
    # the binding's rows started elsewhere in their 16 bytes: other chunks, the same answer
    wide = torch.empty((6, V + 5), dtype=x.dtype, device="cuda")
    wide[:, 3:V + 3] = x.cuda()
    s = g.token_logprobs(wide[:, 3:V + 3], torch.zeros(6, dtype=torch.int64, device="cuda"), top=K)
    assert torch.equal(s["top_id"], r["top_id"])


def _time(x, tok, K):
    ts = []
    for _ in range(7):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(5):
            g.token_logprobs(x, tok, top=K)
        b.record()
        torch.cuda.synchronize()
        ts.append(a.elapsed_time(b))
    return sorted(ts)[3]


@pytest.mark.parametrize("mask", ["inf", "lowest"])
@pytest.mark.parametrize("M,V,K", [(1024, 32000, 5), (64, 128000, 20)])
def test_masks_cost_little(M, V, K, mask):
    """A chunk that is ruled out is read once or twice more, not the fifty times
    of a search: at most the time of four readings (24 times were the search's)."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((M, V), generator=gen, device="cuda")
    tok = torch.zeros(M, dtype=torch.int64, device="cuda")
    value = -float("inf") if mask == "inf" else LOWEST["f32"]
    block, few = x.clone(), torch.full_like(x, value)
    block[:, 8192:16384] = value
    at = torch.randperm(V, generator=gen, device="cuda")[:100]
    few[:, at] = x[:, at]
    plain = _time(x, tok, K)
    for y in (block, few):
        assert _time(y, tok, K) <= 4 * plain
