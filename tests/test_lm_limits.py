"""Limits of the operators around the recurrence: what a call whose dimensions
lie past them answers, on the CPU, before anything is enqueued."""
import pytest

pytest.importorskip("torch")

import gru_recurrence_amd as g  # noqa: E402
from gru_recurrence_amd import lm  # noqa: E402

FAKE = 0x7F0000000000  # never dereferenced: the calls below are refused
UNS = g.RNN_ERR_UNSUPPORTED
BIG = 1 << 60


def _seq():
    return lm._Seq(FAKE, 64, 64)


def _lin_bwd(dims, dt):
    return lm.load().rnn_linattn_bwd(dims, dt, _seq(), _seq(), _seq(), FAKE, 1.0, None, _seq(), None,
                                     FAKE, FAKE, FAKE, None, FAKE, BIG, None)


@pytest.mark.parametrize("dt", [g.RNN_F32, g.RNN_BF16])
@pytest.mark.parametrize("B,NH,NKV,Dk,Dv", [
    (16384, 64, 64, 128, 128), (281250, 16, 16, 16, 16), (1 << 20, 1, 1, 64, 8),
    (1 << 18, 4, 2, 8, 64)])
@pytest.mark.parametrize("T", [1, 2])
def test_linattn_bwd_rows_past_32_bits(T, B, NH, NKV, Dk, Dv, dt):
    """The backward addresses 16 rows of a sequence by 32-bit distances whatever
    the number of tokens; a single token is no exception there."""
    d = lm.LinDims(T, B, NH, NKV, Dk, Dv)
    assert B * NH * max(Dk, Dv) >= 1 << 26
    assert _lin_bwd(d, dt) == UNS
    assert g.workspace_size_linattn(g.OP_LIN_BWD, d, dt) == 0
