"""The binding of the operators around the recurrence: how its functions take
their arguments, on the CPU."""
import inspect

import pytest

torch = pytest.importorskip("torch")

import gru_recurrence_amd as g  # noqa: E402

OPS = ("embed_fwd", "embed_bwd", "token_logprobs", "token_logprobs_bwd", "linattn_fwd",
       "linattn_step", "linattn_bwd")


def _args(op):
    q, ids = torch.zeros((1, 2, 1, 8)), torch.zeros((1, 2), dtype=torch.int64)
    lin = dict(q=q, k=q, v=q, g=torch.zeros(1))
    return {"embed_fwd": dict(ids=ids, table=torch.zeros((5, 8))),
            "embed_bwd": dict(ids=ids, dx=torch.zeros((1, 2, 8)), V=5),
            "token_logprobs": dict(logits=torch.zeros((1, 2, 8)), tokens=ids),
            "token_logprobs_bwd": dict(logits=torch.zeros((1, 2, 8)), tokens=ids,
                                       lse=torch.zeros((1, 2))),
            "linattn_fwd": lin, "linattn_step": dict(lin, S=torch.zeros((2, 1, 8, 8))),
            "linattn_bwd": dict(lin, do=q)}[op]


@pytest.mark.parametrize("op", OPS)
def test_operands_by_name(op):
    """Every operand may be passed by its documented name: what refuses these
    calls is that their tensors are the host's."""
    a = _args(op)
    with pytest.raises(ValueError, match="device tensor"):
        getattr(g, op)(**a)
    first, *rest = a.values()
    with pytest.raises(ValueError, match="device tensor"):
        getattr(g, op)(first, *rest)


@pytest.mark.parametrize("op", OPS)
def test_signature_and_missing_operands(op):
    names = list(inspect.signature(getattr(g, op)).parameters)
    assert names[:len(_args(op))] == list(_args(op))
    with pytest.raises(TypeError, match=names[0]):
        getattr(g, op)()


@pytest.mark.parametrize("op", OPS)
def test_stream_of_another_device(op):
    """A stream that is not the operands' device's is refused: the work would
    go to the other device's current stream, unordered with the caller's."""
    class Stream:
        device = torch.device("cuda", 1)

    class Operand:
        device, is_cuda = torch.device("cuda", 0), True
    rest = list(_args(op).values())[1:]
    with pytest.raises(ValueError, match="stream"):
        getattr(g, op)(Operand(), *rest, stream=Stream())
