"""Verification of drafted tokens against its 64-bit definition: whole numbers, so
equal.  (A draw can differ only where the uniform number falls within about 1e-13
of the sum of a border, one in 10^8 here.)"""
import numpy as np
import pytest

from tests import gated_ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gru_recurrence_amd as g  # noqa: E402

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _case(seed, K, B, V, dt, kind="plain"):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((K + 1, B, V)) * 2
    y = x[:K] + rng.standard_normal((K, B, V)) * 0.6
    if kind == "banned":
        ban = rng.random((K + 1, B, V)) < 0.7
        ban[..., V // 2] = False
        x[ban] = -np.inf
        y[rng.random((K, B, V)) < 0.5] = -np.inf
        x[-1, 0] = -np.inf                       # a row with nothing allowed
        if K:
            y[0, -1] = -np.inf                   # a draft row with nothing allowed
    elif kind == "lowest":
        low = float(torch.finfo(DT[dt]).min)
        x[rng.random((K + 1, B, V)) < 0.5] = low
        y[rng.random((K, B, V)) < 0.5] = low
    elif kind == "peaked":
        x *= 10
        y = x[:K] + rng.standard_normal((K, B, V)) * 0.1
    elif kind == "equal":
        y = x[:K].copy()                         # the same model twice: all accepted
    x, y = (torch.from_numpy(t.astype(np.float32)).to(DT[dt]).cuda() for t in (x, y))
    d = torch.where(torch.rand((K, B)) < 0.7, y.float().argmax(-1).cpu(),
                    torch.from_numpy(rng.integers(0, V, (K, B)))).cuda()
    u = torch.from_numpy(rng.random((K + 1, B)).astype(np.float32)).cuda()
    temp = torch.from_numpy(rng.choice([0.0, -1.0, 0.3, 0.9, 1.7], B).astype(np.float32)).cuda()
    n = torch.from_numpy(rng.integers(0, K + 1, B).astype(np.int32)).cuda()
    return x, d, u, y, temp, n


def _check(x, d, u, y=None, temp=None, n=None, **kw):
    tokens, accepted = g.verify_drafts(x, d, u, y, temperature=temp, n_drafts=n, **kw)
    assert tokens.dtype == torch.int32 and accepted.dtype == torch.int32
    rt, ra = gated_ref.verify(_np(x), d.cpu().numpy(), _np(u), _np(y), _np(temp),
                              None if n is None else n.cpu().numpy())
    assert np.array_equal(accepted.cpu().numpy(), ra), (accepted, ra)
    assert np.array_equal(tokens.cpu().numpy(), rt), (tokens.cpu().numpy(), rt)
    return tokens, accepted


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["plain", "banned", "lowest", "peaked", "equal"])
@pytest.mark.parametrize("K,B,V", [(0, 3, 5), (1, 1, 1), (1, 4, 2), (2, 3, 65), (4, 5, 1000), (7, 6, 4097),
                                   (3, 2, 4096), (5, 3, 20011), (63, 2, 130), (1, 40, 333)])
def test_verify(K, B, V, kind, dt):
    torch.manual_seed(K + V)
    x, d, u, y, temp, n = _case(K * 1000 + V, K, B, V, dt, kind)
    for q in (y, None):
        _check(x, d, u, q)
        _check(x, d, u, q, temp)
        _check(x, d.int(), u, q, None, n)
        _check(x, d, u, q, temp, n)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_verify_every_uniform_number(dt):
    """One row, uniform numbers over the whole of [0, 1]."""
    torch.manual_seed(0)
    B, V = 4000, 50
    x, _, _, y, _, _ = _case(3, 1, 1, V, dt)
    x, y = x.expand(2, B, V), y.expand(1, B, V)
    d = torch.randint(0, V, (1, B), device="cuda")
    u = torch.linspace(0, 1, B, device="cuda").repeat(2, 1)
    u[0] = torch.rand(B, device="cuda")
    _check(x, d, u, y)
    _check(x, d, u)
    _check(x[1:], d[:0], u[1:])


def test_verify_equal_weights():
    """Equal logits: every weight is exactly 1, so that a uniform number on a border
    belongs to the entry above it."""
    V = 8192
    x = torch.full((1, V + 1, V), 0.3, device="cuda")
    u = (torch.arange(V + 1, device="cuda") / V)[None].float()
    tokens, _ = g.verify_drafts(x, None, u)
    want = torch.arange(V + 1, device="cuda").clamp(max=V - 1)
    assert torch.equal(tokens[0].long(), want)


def test_verify_greedy_ties_and_lookup():
    V = 9000
    x = torch.zeros((3, 2, V), device="cuda")
    x[0, :, 5000], x[0, :, 8999] = 1.0, 1.0
    x[1, :, :] = -0.0
    x[1, 0, 3] = 0.0
    zero = torch.zeros(2, device="cuda")
    u = torch.full((3, 2), 0.999, device="cuda")
    d = torch.tensor([[5000, 8999], [0, 0]], device="cuda")
    tokens, acc = g.verify_drafts(x, d, u, temperature=zero)
    assert acc.tolist() == [2, 0] and tokens[:, 0].tolist() == [5000, 0, 0]
    assert tokens[:, 1].tolist() == [5000, -1, -1]


def test_verify_outside_and_not_finite():
    torch.manual_seed(1)
    x, d, u, y, temp, _ = _case(9, 3, 6, 5000, "f32")
    d[0, 0], d[1, 1], d[2, 2] = -1, 5000, 1 << 40
    _check(x, d, u, y)
    _check(x, d, u)
    nan, inf = float("nan"), float("inf")
    x[1, 0, 17], x[0, 1, 4500], x[3, 2, 0], x[0, 3, :] = nan, inf, nan, nan
    y[0, 4, 9], y[1, 5, 4999] = nan, inf
    u[0, 5], u[3, 5], u[1, 4] = nan, -0.5, 2.0
    _check(x, d, u, y)
    _check(x, d, u, y, temp)
    _check(x, d, u)
    _check(x, d, u, y, torch.tensor([inf, 1e-30, 1e30, 1e-45, nan, 1.0], device="cuda"))
    n = torch.tensor([-3, 0, 1, 3, 99, 2], dtype=torch.int32, device="cuda")
    _check(x, d, u, y, None, n)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_verify_views(dt):
    """Batch-first logits, padded vocabularies, rows that start anywhere and differ
    between the two models, transposed drafts."""
    torch.manual_seed(2)
    K, B, V = 4, 5, 5001
    x, d, u, y, temp, n = _case(21, K, B, V, dt)
    want = _check(x, d, u, y, temp, n)
    xb = x.transpose(0, 1).contiguous().transpose(0, 1)
    for lo, hi in ((0, 0), (1, 3), (5, 2)):
        xp = torch.nn.functional.pad(x, (lo, hi), value=50.0)[..., lo:lo + V]
        yp = torch.nn.functional.pad(y, (hi, lo), value=50.0)[..., hi:hi + V]
        for a, b in ((xp, y), (x, yp), (xp, yp), (xb, yp)):
            got = g.verify_drafts(a, d.t().contiguous().t(), u, b, temperature=temp, n_drafts=n)
            assert all(torch.equal(s, t) for s, t in zip(got, want))


def test_verify_rows_behind_the_drafts_are_not_read():
    torch.manual_seed(3)
    x, d, u, y, _, n = _case(33, 5, 8, 6000, "f32")
    want = g.verify_drafts(x, d, u, y, n_drafts=n)
    for b, k in enumerate(n.tolist()):
        x[k + 1:, b], y[k:, b], d[k:, b], u[k:5, b] = float("nan"), float("nan"), 1 << 50, float("nan")
    got = g.verify_drafts(x, d, u, y, n_drafts=n)
    assert all(torch.equal(s, t) for s, t in zip(got, want))


def test_verify_large_vocabularies_and_offsets_past_32_bits():
    torch.manual_seed(4)
    for V, dt in ((1000000, "bf16"), (128001, "f32")):
        x, d, u, y, temp, _ = _case(V, 2, 2, V, dt)
        _check(x, d, u, y)
        _check(x, d, u, None, temp)
    B, V = 60000, 40001  # 2.4e9 logits
    x = torch.zeros((1, B, V), dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([0, 53686, 53688, B - 1], device="cuda")
    z, _, _, _, _, _ = _case(1, 0, 4, V, "bf16")
    x[0, rows] = z[0]
    u = torch.rand((1, B), device="cuda")
    tokens, _ = g.verify_drafts(x, None, u)
    want, _ = g.verify_drafts(z, None, u[:, rows].contiguous())
    assert torch.equal(tokens[:, rows], want)
    rest = torch.ones(B, dtype=torch.bool, device="cuda")
    rest[rows] = False
    # equal weights: entry floor(u V)
    flat = torch.floor(u[0].double() * V).int()
    assert torch.equal(tokens[0, rest], flat[rest])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_verify_large_calls(dt):
    """Calls large enough for the longer chunks, with a mask and temperatures; rows of
    the two models that start at the same place of their 16 bytes, and elsewhere."""
    torch.manual_seed(8)
    K, B, V = 4, 40, 100003
    x, d, u, y, temp, n = _case(77, K, B, V, dt, "banned")
    want = _check(x, d, u, y, temp, n)
    _check(x, d, u, None, temp)
    yp = torch.nn.functional.pad(y, (3, 0))[..., 3:]
    got = g.verify_drafts(x, d, u, yp, temperature=temp, n_drafts=n)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["plain", "banned", "peaked", "equal"])
@pytest.mark.parametrize("K", [0, 2])
def test_verify_many_sequences(K, kind, dt):
    """Enough sequences that a row of p is left to one workgroup; every place of u."""
    B, V = 400, 9001
    x, d, u, y, temp, n = _case(K + 31, K, B, V, dt, kind)
    u[K] = torch.linspace(0.0, 1.0, B)
    u[K, -1] = 1.0 - 2.0 ** -24
    _check(x, d, u, y, temp, n)
    _check(x, d, u, None, temp, n)
    _check(x, d, u, y if K else None)


@pytest.mark.parametrize("V", [7, 5000, 70001])
def test_verify_nothing_left_of_the_difference(V):
    """The same model twice and u = 1: every draft is refused, max(p - q, 0) is 0
    everywhere, and p itself is drawn from."""
    torch.manual_seed(9)
    x, d, u, y, _, _ = _case(V, 2, 9, V, "f32", "equal")
    u[:2] = 1.0
    tokens, acc = _check(x, d, u, y)
    assert not acc.any()
    want, _ = g.verify_drafts(x[:1], None, u[2:])
    assert torch.equal(tokens[:1], want)


def test_verify_is_distributed_as_the_target():
    """Drafts drawn from q and verified against p: the first token that comes out
    is distributed as p, whatever q is.  Counts of n draws stay within 5 of their
    standard deviations sqrt(n p (1 - p))."""
    torch.manual_seed(5)
    B, V = 200000, 12
    x = torch.randn((2, 1, V), device="cuda") * 1.5
    y = torch.randn((1, 1, V), device="cuda") * 1.5
    d = torch.multinomial(torch.softmax(y[0, 0] / 0.8, -1), B, replacement=True)[None]
    u = torch.rand((2, B), device="cuda")
    t = torch.full((B,), 0.8, device="cuda")
    tokens, acc = g.verify_drafts(x.expand(2, B, V), d, u, y.expand(1, B, V), temperature=t)
    p = torch.softmax(x[0, 0].double() / 0.8, -1)
    n = torch.bincount(tokens[0].long(), minlength=V).double()
    assert ((n - B * p).abs() <= 5 * (B * p * (1 - p)).sqrt() + 1).all()
    q = torch.softmax(y[0, 0].double() / 0.8, -1)
    share = torch.minimum(p, q).sum().item()
    assert abs(acc.double().mean().item() - share) <= 5 * (share * (1 - share) / B) ** 0.5


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_verify_stream_and_graph(dt):
    torch.manual_seed(6)
    K, B, V = 4, 7, 20011
    x, d, u, y, temp, n = _case(55, K, B, V, dt)
    ws = torch.empty(g.workspace_size_verify(K, B, V), dtype=torch.uint8, device="cuda")
    want = _check(x, d, u, y, temp, n)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(4):
        side.wait_stream(torch.cuda.current_stream())
        got = g.verify_drafts(x, d, u, y, temperature=temp, n_drafts=n, stream=side)
        torch.full((1 << 20,), 7.0, device="cuda")
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = g.verify_drafts(x, d, u, y, temperature=temp, n_drafts=n, ws=ws)
    for i in range(4):
        x.copy_(x.roll(i, 2))
        y.copy_(y.roll(i, 2))
        u.copy_(u.roll(1, 1))
        graph.replay()
        got = [t.clone() for t in out]
        for a, b in zip(got, g.verify_drafts(x, d, u, y, temperature=temp, n_drafts=n)):
            assert torch.equal(a, b), i
        torch.cuda.synchronize()


def test_state_goes_back_to_the_accepted_part():
    """The operators together, as a server uses them: the recurrence runs over the
    drafted tokens, the drafts are verified, and the state is taken back to the
    last token that stands, with lens = accepted + 1."""
    torch.manual_seed(7)
    K, B, D, V = 4, 6, 32, 500
    E, W = torch.randn((V, 2 * D), device="cuda"), torch.randn((D, V), device="cuda")
    h0 = torch.randn((B, D), device="cuda")
    ids = torch.randint(0, V, (K + 1, B), device="cuda")  # last token, then the drafts
    f, x = g.embed_fwd(ids, E).split(D, -1)
    h, _ = g.gated_fwd(f, x, h0)
    logits = g.input_proj(h, W)
    tokens, acc = g.verify_drafts(logits, ids[1:], torch.rand((K + 1, B), device="cuda"))
    _, S = g.gated_fwd(f, x, h0, lens=acc + 1)
    for b, k in enumerate(acc.tolist()):
        assert tokens[:k, b].tolist() == ids[1:k + 1, b].tolist()
        want = h0[b:b + 1].contiguous()
        for t in range(k + 1):
            _, want = g.gated_step(f[t:t + 1, b:b + 1], x[t:t + 1, b:b + 1], want.clone())
        assert (S[b] - want[0]).abs().max() <= 1e-5
