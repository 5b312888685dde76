"""The example language model: the operators together, trained and decoded."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location(
        "recurrent_lm", os.path.join(ROOT, "examples", "recurrent_lm.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_gradients_of_the_whole_model_by_differences():
    ex = _example()
    m = ex.RecurrentLM(vocab=32, heads=2, head_dim=16)
    ids, targets = ex.text(24, 3, m.V)
    targets[3, 1] = -1  # a token that is not scored
    _, d = m.gradients(ids, targets)
    torch.manual_seed(0)
    for n in ("E", "W", "R", "b", "Wqkv", "Wout"):
        v = torch.randn_like(m.p[n])
        v /= v.norm()
        h, keep = 2e-2, m.p[n].clone()
        out = []
        for s in (h, -h):
            m.p[n] = keep + s * v
            out.append(m.gradients(ids, targets)[0].double().item())
        m.p[n] = keep
        num, ana = (out[0] - out[1]) / (2 * h), (d[n].double() * v.double()).sum().item()
        # h^2 times a third derivative of order the gradient's norm, and 1e-7 / h of rounding
        assert abs(num - ana) <= 4 * h * h * d[n].norm().item() + 3e-5, (n, num, ana)


def test_training_lowers_the_loss_and_decoding_follows_the_text():
    ex = _example()
    m = ex.RecurrentLM()
    ids, targets = ex.text(96, 8, m.V)
    losses = m.train(ids, targets, 60)
    assert losses[0] > 3.5 and losses[-1] < 0.5 * losses[0], losses[::10]
    # token by token from the prompt's state gives what one pass over all gives
    full, _, _ = m.forward(ids[:60])
    part, _, state = m.forward(ids[:40])
    rows = [part]
    for t in range(40, 60):
        l, _, state = m.forward(ids[t:t + 1], state)
        rows.append(l)
    got = torch.cat(rows)
    assert (got - full).norm() <= 1e-4 * full.norm()
    out, lp = m.generate(ids[:40], 8)
    assert out.shape == (8, 8) and (lp <= 0).all()
