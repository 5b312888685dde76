"""The example model of gated recurrences: the operators together, trained and
decoded with drafted tokens."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location(
        "gated_lm", os.path.join(ROOT, "examples", "gated_lm.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_gradients_of_the_whole_model_by_differences():
    ex = _example()
    m = ex.GatedLM(vocab=32, width=32)
    ids, targets = ex.text(150, 3, m.V)  # longer than a segment
    targets[3, 1] = -1  # a token that is not scored
    _, d = m.gradients(ids, targets)
    assert sorted(d) == sorted(m.p)
    torch.manual_seed(0)
    for n in d:
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


def test_trains_and_continues_with_drafts():
    ex = _example()
    m = ex.GatedLM()
    ids, targets = ex.text(96, 8, m.V)
    losses = m.train(ids, targets, 20)
    assert len(losses) == 20 and all(x == x for x in losses)
    # one pass over all gives what token by token from the prompt's states gives
    full, _, _ = m.forward(ids[:60])
    part, _, states = m.forward(ids[:40])
    rows = [part]
    for t in range(40, 60):
        l, _, states = m.forward(ids[t:t + 1], states)
        rows.append(l)
    assert (torch.cat(rows) - full).norm() <= 1e-5 * full.norm()
    # greedy: the drafts change how many passes it takes, not what comes out
    want = m.generate(ids[:40], 24).t().tolist()
    out, passes = m.continue_drafted(ids[:40], 24)
    assert [t[:24] for t in out] == want
    assert passes <= 24
    out, _ = m.continue_drafted(ids[:40], 10, drafts=7, temperature=0.9)
    assert all(len(t) >= 10 and all(0 <= x < m.V for x in t) for t in out)
