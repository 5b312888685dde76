"""Ends of the ranges of the gated recurrence, gradient clipping and draft
verification: what their workspaces report, values near float32's largest, logits
that are infinite, roundings next to a border, equal rows at different places."""
import numpy as np
import pytest

from tests import gated_ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gru_recurrence_amd as g  # noqa: E402
from tests.test_gpu_gated import _np, _within  # noqa: E402

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _odd(t):
    """The same values in rows that start at an odd element."""
    return torch.nn.functional.pad(t, (1, 2 - t.shape[-1] % 2))[..., 1:t.shape[-1] + 1]


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("T,B,D", [(1024, 16, 768), (600, 24, 500), (100, 32, 700), (300, 10, 1024)])
def test_gated_status_is_ok_on_a_workspace_holding_garbage(T, B, D, odd):
    """Whatever plan the operands' alignment gives a call that asks for a workspace,
    it leaves the status word of that call there."""
    gen = torch.Generator(device="cuda").manual_seed(T)
    f, x, dh = (torch.randn((T, B, D), generator=gen, device="cuda").bfloat16() for _ in range(3))
    if odd:
        f, x, dh = _odd(f), _odd(x), _odd(dh)
    d = g.GatedDims(T, B, D)
    need = [g.workspace_size_gated(op, d, g.RNN_BF16) for op in (g.OP_GATED_FWD, g.OP_GATED_BWD)]
    assert max(need) > 0
    h, _ = g.gated_fwd(f, x)
    for n, call in zip(need, (lambda w: g.gated_fwd(f, x, ws=w), lambda w: g.gated_bwd(f, x, h, dh, ws=w))):
        if n == 0:
            continue
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        call(ws)
        assert g.workspace_status(ws) == g.RNN_OK
