"""Gradient norm and clipping against 64 bits.  Squares and their sum are 64-bit,
so the norm is off by its rounding to float32, u = 2^-24 relative; a clipped value
by three roundings, 3 u: the bound's on its way in (the call takes a float32, these
tests compute with the double: value = g fl(fl(bound) / norm), each fl within u),
the factor's and the product's; and its rounding to bf16, 2^-8."""
import numpy as np
import pytest

from tests import gated_ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gru_recurrence_amd as g  # noqa: E402

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _np(t):
    return t.detach().double().cpu().numpy()


def _grads(seed, sizes, dts, std=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=gen, device="cuda") * std).to(DT[dts[i % len(dts)]])
            for i, n in enumerate(sizes)]


def _check(grads, max_norm, out=None, inplace=False):
    norm, ref = gated_ref.clip([_np(t) for t in grads], max_norm)
    keep = [t.clone() for t in grads]
    got = g.clip_grads(grads, max_norm, out=out)
    assert got.shape == () and got.dtype == torch.float32
    assert abs(got.item() - norm) <= (U + 1e-12) * norm, (got.item(), norm)
    for t, k, o, r in zip(grads, keep, grads if out is None else out, ref):
        if out is not None:
            assert torch.equal(t, k)
        r = np.asarray(r)
        err = np.abs(_np(o) - r)
        lim = (3 * U + (2.0 ** -8 if o.dtype == torch.bfloat16 else 0.0)) * 1.001 * np.abs(r) + 1e-40
        if norm <= max_norm:
            assert torch.equal(o, k)
        assert (err <= lim).all()
    return got


SIZES = [[(1,)], [(3,), (5, 7), (1, 1, 1)], [(0,), (4,), (0, 5)], [(4096,), (4097,), (12345,)],
         [(1000, 33), (8, 1024), (129,)], [(300000,), (1,), (70000, 3)],
         [(int(n),) for n in np.random.default_rng(0).integers(0, 3000, 230)]]


@pytest.mark.parametrize("dts", [["f32"], ["bf16"], ["f32", "bf16"]], ids=str)
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "%d tensors" % len(s))
def test_clip(sizes, dts):
    grads = _grads(len(sizes), sizes, dts)
    norm = float(np.sqrt(sum((_np(t) ** 2).sum() for t in grads)))
    n = g.grad_norm(grads)
    assert abs(n.item() - norm) <= (U + 1e-12) * norm
    for share in (0.37, 1.5):
        out = [torch.full_like(t, 7.0) for t in grads]
        _check(grads, share * norm, out)
        a = _check([t.clone() for t in grads], share * norm)
        assert a.item() == n.item()  # the same sum in the same order


def test_clip_repeats_bit_for_bit():
    grads = _grads(3, [(1 << 20,), (777,), (50000,)], ["f32", "bf16"])
    first = g.grad_norm(grads)
    for _ in range(5):
        assert torch.equal(g.grad_norm(grads), first)


def test_clip_any_start():
    """Tensors that start at any element, outputs that start elsewhere."""
    big, other = _grads(1, [(40000,), (40000,)], ["f32"])
    for dt in (torch.float32, torch.bfloat16):
        a, b = big.to(dt), other.to(dt)
        for i, j, n in ((1, 1, 9000), (1, 2, 9000), (3, 0, 20001), (7, 5, 1), (2, 2, 5), (5, 9, 4099)):
            b.fill_(7.0)
            _check([a[i:i + n], a[20:23]], 1.0, [b[j:j + n], b[39000:39003]])
            assert (b[:j] == 7).all() and (b[j + n:39000] == 7).all() and (b[39003:] == 7).all()


def test_clip_limits():
    grads = _grads(2, [(1000,), (20,)], ["f32"])
    out = [torch.full_like(t, 7.0) for t in grads]
    assert g.clip_grads(grads, 0.0, out=out) > 0
    assert not any(t.any() for t in out)
    zero = [torch.zeros(5, device="cuda"), torch.zeros((0, 3), device="cuda")]
    assert g.clip_grads(zero, 0.0).item() == 0 and not zero[0].any()
    assert g.grad_norm([torch.zeros(0, device="cuda")]).item() == 0
    # an infinite bound clips nothing
    keep = [t.clone() for t in grads]
    g.clip_grads(grads, float("inf"))
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))
    # values whose squares leave float32, at either end
    for v in (1e30, 1e-30):
        t = torch.full((300,), v, device="cuda")
        n = g.clip_grads([t], v)
        # the norm is v' sqrt(300) with v' the float32 next to v
        want = float(np.float32(v)) * np.sqrt(300)
        assert abs(n.item() - want) <= U * 1.001 * want
        assert (t.double() - v / np.sqrt(300)).abs().max() <= 4 * U * v / np.sqrt(300)
    # a norm past float32 is inf and clips all the same
    t = torch.full((300,), 3e38, device="cuda")
    assert g.clip_grads([t], 1.0).item() == float("inf")
    assert (t.double() * np.sqrt(300) - 1.0).abs().max() <= 4 * U
    # subnormal gradients
    t = torch.full((10,), 1e-41, device="cuda")
    n = g.grad_norm([t]).item()
    assert abs(n - t[0].double().item() * np.sqrt(10)) <= 2e-45


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_clip_not_finite(bad, dt):
    """A norm that is not finite leaves everything as it is."""
    grads = _grads(4, [(5000,), (33,)], [dt])
    grads[1][32] = bad
    out = [torch.full_like(t, 7.0) for t in grads]
    n = g.clip_grads(grads, 0.1, out=out)
    assert torch.isnan(n) if bad != bad else n.item() == float("inf")
    for a, b in zip(grads, out):
        assert torch.equal(torch.nan_to_num(a, nan=5.0), torch.nan_to_num(b, nan=5.0))
    keep = [t.clone() for t in grads]
    g.clip_grads(grads, 0.1)
    for a, b in zip(grads, keep):
        assert torch.equal(torch.nan_to_num(a, nan=5.0), torch.nan_to_num(b, nan=5.0))


def test_clip_past_32_bits():
    t = torch.zeros((1 << 32) + 77, dtype=torch.bfloat16, device="cuda")
    t[-1], t[1 << 31], t[5] = 3.0, 4.0, 12.0
    n = g.clip_grads([t, torch.zeros(3, device="cuda")], 6.5)
    assert n.item() == 13.0
    assert t[-1].item() == 1.5 and t[1 << 31].item() == 2.0 and t[5].item() == 6.0
    assert t.count_nonzero().item() == 3


def test_clip_list_kept():
    grads = _grads(6, [(300, 7), (11,)], ["f32", "bf16"])
    out = [torch.empty_like(t) for t in grads]
    lst = g.GradList(grads, out)
    for i in range(3):
        for t in grads:
            t.mul_(1.0 + i)
        n = g.clip_grads(lst, 2.0)
        want = [torch.empty_like(t) for t in grads]
        assert torch.equal(n, g.clip_grads(grads, 2.0, out=want))
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_clip_stream_and_graph():
    sizes = [(1 << 18,), (513, 9), (7,)] + [(100 + i,) for i in range(120)]
    grads = _grads(7, sizes, ["f32", "bf16"])
    out = [torch.empty_like(t) for t in grads]
    ws = torch.empty(g.workspace_size_clip(grads), dtype=torch.uint8, device="cuda")
    want = g.clip_grads(grads, 1.0, out=out)
    ref = [t.clone() for t in out]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        for t in out:
            t.zero_()
        side.wait_stream(torch.cuda.current_stream())
        n = g.clip_grads(grads, 1.0, out=out, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(n, want) and all(torch.equal(a, b) for a, b in zip(out, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n = g.clip_grads(grads, 1.0, out=out, ws=ws)
    for i in range(4):
        for t in grads:
            t.mul_(0.5 + i)
        graph.replay()
        got = [n.clone()] + [t.clone() for t in out]
        eager = [torch.empty_like(t) for t in grads]
        assert torch.equal(got[0], g.clip_grads(grads, 1.0, out=eager)), i
        assert all(torch.equal(a, b) for a, b in zip(got[1:], eager)), i
        torch.cuda.synchronize()


@pytest.mark.parametrize("dts", [["f32"], ["bf16"]], ids=str)
@pytest.mark.parametrize("sizes", [[(777,), (31,)], [(300000,), (1,), (70000, 3)]], ids=str)
def test_clip_factor_below_float32(sizes, dts):
    """Values of 1e37 clipped to a norm of 1e-3: the factor, some 1e-42, is below
    float32's normal numbers, where it would have ten bits; the results are not."""
    grads = _grads(9, sizes, dts, 1e37)
    norm, ref = gated_ref.clip([_np(t) for t in grads], 1e-3)
    with np.errstate(over="ignore"):
        want = float(np.float32(norm))  # +inf where float32 ends
    got = g.clip_grads(grads, 1e-3).item()
    assert got == want or abs(got - norm) <= (U + 1e-12) * norm, (got, norm)
    for o, r in zip(grads, ref):
        lim = (3 * U + (2.0 ** -8 if o.dtype == torch.bfloat16 else 0.0)) * 1.001 * np.abs(r) + 1e-40
        assert (np.abs(_np(o) - r) <= lim).all()
