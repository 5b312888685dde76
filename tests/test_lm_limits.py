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


def test_launches_past_2_32_threads():
    """A launch has fewer than 2^32 threads in a dimension; calls that would
    need more say so instead of failing at the launch, or between two."""
    lib = lm.load()
    ids = lm._Ids(FAKE, 0, 1, 1)
    assert lib.rnn_embed_fwd(1 << 15, 1 << 14, 100, 8, 1, ids, FAKE, 8, 1.0, FAKE, None) == UNS
    assert lib.rnn_embed_fwd(1 << 13, 1 << 13, 100, 256, 0, ids, FAKE, 256, 1.0, FAKE, None) == UNS
    assert lib.rnn_embed_bwd(1 << 15, 1 << 15, 1 << 30, 1, 0, ids, FAKE, 1.0, FAKE, FAKE, BIG, None) == UNS

    def logp(M, V, dt):
        return lib.rnn_token_logprobs(M, V, dt, FAKE, V, FAKE, 0, 0, FAKE, None, None, None, None, FAKE,
                                      BIG, None)

    def logp_bwd(M, V, dt):
        return lib.rnn_token_logprobs_bwd(M, V, dt, FAKE, V, FAKE, 0, FAKE, None, FAKE, None, FAKE, V, None)
    for dt in (0, 1):
        assert logp(1 << 24, 10, dt) == UNS and logp(1 << 23, 8194, dt) == UNS
        assert logp_bwd(1 << 24, 10, dt) == UNS and logp_bwd(1 << 22, 32768, dt) == UNS

        one = lm.LinDims(1, 1 << 20, 16, 16, 1, 1)
        s = [_seq()] * 3
        assert lib.rnn_linattn_step(one, dt, *s, FAKE, 1.0, FAKE, FAKE, FAKE, None) == UNS
        for T in (1, 2):
            d = lm.LinDims(T, 1 << 20, 16, 16, 1, 1)
            assert lib.rnn_linattn_fwd(d, dt, *s, FAKE, 1.0, None, FAKE, FAKE, FAKE, BIG, None) == UNS
        for d in (lm.LinDims(2, 1 << 19, 16, 16, 1, 1), lm.LinDims(2, 1 << 19, 16, 16, 1, 2),
                  lm.LinDims(1 << 20, 1 << 10, 4, 2, 32, 32)):
            assert _lin_bwd(d, dt) == UNS
