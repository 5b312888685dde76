"""Linear attention's general form (rows at odd elements, widths that are no
whole tiles) over long sequences: many segments, in pieces, with the carry in a
launch of its own; against the 64-bit definition with the bounds of the other
shapes."""
import pytest

pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests import test_gpu_lm as base  # noqa: E402


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,B,NH,NKV,Dk,Dv", [
    (4001, 1, 1, 1, 33, 70), (2500, 1, 2, 1, 20, 20), (3000, 1, 1, 1, 130, 40), (2049, 2, 2, 2, 64, 100)])
def test_many_segments(T, B, NH, NKV, Dk, Dv, dt):
    base._check_lin(T, B, NH, NKV, Dk, Dv, dt, "odd")
