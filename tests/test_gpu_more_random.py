"""Seeded random calls of the gated recurrence, gradient clipping and draft
verification: sizes, types, layouts, lengths and options drawn together, against
the 64-bit definitions within the bounds of the operators' own tests."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests import test_gpu_clip, test_gpu_gated, test_gpu_verify  # noqa: E402


def _log(rng, lo, hi):
    return int(round(float(np.exp(rng.uniform(np.log(lo), np.log(hi))))))


@pytest.mark.parametrize("seed", range(24))
def test_gated(seed):
    rng = np.random.default_rng(1000 + seed)
    D, B = _log(rng, 1, 300), _log(rng, 1, 20)
    T = min(_log(rng, 1, 4000), 400000 // (B * D) + 1)
    test_gpu_gated._check(T, B, D, rng.choice(["bf16", "f32"]), rng.choice(["logit", "decay"]),
                          rng.choice(["dense", "fused", "bt", "odd"]), bool(rng.random() < 0.4),
                          bool(rng.random() < 0.6), seed)


@pytest.mark.parametrize("seed", range(12))
def test_clip(seed):
    rng = np.random.default_rng(2000 + seed)
    sizes = [(_log(rng, 1, 60000),) for _ in range(_log(rng, 1, 250))]
    dts = [["f32"], ["bf16"], ["bf16", "f32", "f32"]][seed % 3]
    grads = test_gpu_clip._grads(seed, sizes, dts, float(np.exp(rng.uniform(-12, 6))))
    norm = float(np.sqrt(sum((test_gpu_clip._np(t) ** 2).sum() for t in grads)))
    out = [torch.empty_like(t) for t in grads]
    test_gpu_clip._check(grads, float(rng.uniform(0.01, 1.4)) * norm, out if seed % 2 else None)


@pytest.mark.parametrize("seed", range(24))
def test_verify(seed):
    rng = np.random.default_rng(3000 + seed)
    torch.manual_seed(seed)
    K, B, V = int(rng.integers(0, 9)), _log(rng, 1, 24), _log(rng, 1, 30000)
    x, d, u, y, temp, n = test_gpu_verify._case(seed, K, B, V, rng.choice(["bf16", "f32"]),
                                                rng.choice(["plain", "banned", "lowest", "peaked"]))
    if rng.random() < 0.3:
        x = x.transpose(0, 1).contiguous().transpose(0, 1)
    if rng.random() < 0.3:
        lo = int(rng.integers(1, 9))
        y = torch.nn.functional.pad(y, (lo, 3))[..., lo:lo + V]
    test_gpu_verify._check(x, d if rng.random() < 0.5 else d.int(), u, y if rng.random() < 0.6 else None,
                           temp if rng.random() < 0.5 else None, n if rng.random() < 0.5 else None)
