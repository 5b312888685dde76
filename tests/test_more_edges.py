"""Refusals of gradient clipping's overlapping outputs, on the CPU: before anything
is enqueued."""
import pytest

torch = pytest.importorskip("torch")

import gru_recurrence_amd as g  # noqa: E402
from gru_recurrence_amd import lm  # noqa: E402

FAKE = 0x7F0000000000  # never dereferenced: validation fails first
NORM = FAKE - 4096
BIG = 1 << 60


def _list(*rows):
    return (lm._Grad * len(rows))(*rows)


def _far(n):
    """n small tensors, apart from each other and from the others below."""
    return [(FAKE + (1 << 30) + 64 * i, FAKE + (1 << 31) + 64 * i, 16, 0) for i in range(n)]


A, B = FAKE, FAKE + 1024  # 64 float32 or 128 bf16 values take 256 bytes


@pytest.mark.parametrize("more", [0, 3, 300])
@pytest.mark.parametrize("rows", [
    [(A, B, 64, 0), (B, A, 64, 0)],                       # swapped
    [(A, B, 64, 0), (B, None, 64, 0)],                    # over a tensor clipped in place
    [(A, B, 64, 0), (B + 252, FAKE + 8192, 64, 0)],       # the last value is another's first
    [(A, B, 64, 0), (FAKE + 8192, B, 64, 0)],             # the same output twice
    [(A, B, 64, 0), (FAKE + 8192, B - 254, 128, 1)],      # outputs that share two bytes
    [(A, None, 64, 0), (A, None, 64, 0)],                 # in place twice
    [(A, None, 64, 0), (A + 128, B, 1, 1)],               # in place under one that is read
    [(A, A + 4, 64, 0)],                                  # its own values, at another place
    [(A, None, 1 << 20, 0), (A + 16, B, 1, 0), (A + 64, FAKE + 8192, 1, 0)],
    [(NORM - 64, None, 17, 0)],                           # the norm among the values
    [(A, NORM, 64, 0)],                                   # the norm in an output
])
def test_clip_refuses_overlapping_outputs(rows, more):
    lib = lm.load()
    for lst in (rows, rows[::-1]):
        for lst in (lst + _far(more), _far(more) + lst):
            a = _list(*lst)
            assert lib.rnn_clip_grads(len(lst), a, 1.0, NORM, FAKE + (1 << 40), BIG, None) == g.RNN_ERR_INVALID_ARG


def test_states_must_start_at_16_bytes():
    """Rows of a state whose width is no multiple of four values: the library's refusal
    is explained by name, others as they come."""
    many = torch.zeros((5, 129))
    at = [i for i in range(5) if many[i].data_ptr() % 16]
    with pytest.raises(ValueError, match="hT must start.*16 bytes"):
        lm._refused(g.RNN_ERR_INVALID_ARG, "rnn_gated_fwd", h0=None, hT=many[at[0]:at[0] + 1])
    for s, t in ((g.RNN_ERR_INVALID_ARG, None), (g.RNN_ERR_UNSUPPORTED, many[at[0]])):
        with pytest.raises(g.RnnError) as e:
            lm._refused(s, "rnn_gated_fwd", h0=t)
        assert e.value.status == s
