"""Measured cases of the gated linear recurrence (forward, single token,
backward), of the global gradient norm with clipping, and of the verification
of drafted tokens.

Each case has a plain form in elementary torch operations (`own` false), the
library's call (`own` true) and the definition in 64 bits (`exact`)."""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # forward of a layer in training, at the headline's batch and width: gate
        # and input are the halves of one projection
        dict(name="gated t1024 b16", op="gated_fwd", T=1024, B=16, D=768, dt="bf16", gate="logit",
             state=False, layout="fused", ragged=False),
        # one long document carried on from a state, float32
        dict(name="gated long f32", op="gated_fwd", T=32768, B=1, D=768, dt="f32", gate="logit",
             state=True, layout="dense", ragged=False),
        # prompts of different lengths kept batch-first, odd width, decays given as they are
        dict(name="gated prompts ragged", op="gated_fwd", T=777, B=5, D=331, dt="bf16",
             gate="decay", state=True, layout="bt", ragged=True),
        # decoding: 64 sequences, one token each (latency)
        dict(name="gated step b64", op="gated_step", T=1, B=64, D=768, dt="bf16", gate="logit",
             state=True, layout="fused", ragged=False),
        # backward of a training batch, ragged length of the window
        dict(name="gated grad t1000 b16", op="gated_bwd", T=1000, B=16, D=1024, dt="bf16",
             gate="logit", state=True, layout="fused", ragged=False),
        # backward over prompts of different lengths, float32, odd width
        dict(name="gated grad ragged f32", op="gated_bwd", T=301, B=7, D=129, dt="f32",
             gate="decay", state=True, layout="dense", ragged=True),
        # gradients of a language model of four LSTM layers in heads of 256, clipped for the
        # update into buffers of their own
        dict(name="clip model", op="clip", sizes="model", n=0, dt="f32", over=True, inplace=False),
        # a small layer whose norm stays below the bound, in place (latency)
        dict(name="clip small below", op="clip", sizes="layer", n=0, dt="f32", over=False,
             inplace=True),
        # many tensors of any size, bf16
        dict(name="clip many bf16", op="clip", sizes="many", n=60, dt="bf16", over=True,
             inplace=False),
        # one sequence, four drafted tokens, both models' logits (latency)
        dict(name="verify b1 k4", op="verify", B=1, K=4, V=32000, dt="f32", q=True, ragged=False,
             temp="none"),
        # a serving batch with a long vocabulary
        dict(name="verify b32 k4", op="verify", B=32, K=4, V=128000, dt="bf16", q=True,
             ragged=False, temp="same"),
        # drafts looked up in the text (no probabilities of their own), a different number for
        # each sequence, temperatures of their own, some greedy
        dict(name="verify lookup b16 k7", op="verify", B=16, K=7, V=50001, dt="f32", q=False,
             ragged=True, temp="mixed"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated_fwd", "gated_fwd", "gated_step", "gated_bwd", "gated_bwd", "clip",
                     "verify", "verify"])
    dt = rng.choice(["bf16", "f32"])
    if op.startswith("gated"):
        D = rng.choice([1, 64, 100, 129, 331, 512, 768, 1024, 2047])
        B = _log_int(rng, 1, 32)
        T = max(1, min(_log_int(rng, 1, 32768), 16_000_000 // (B * D)))
        if op == "gated_step":
            T, B = 1, _log_int(rng, 1, 256)
        return dict(op=op, T=T, B=B, D=D, dt=dt, gate=rng.choice(["logit", "logit", "decay"]),
                    state=op == "gated_step" or rng.random() < 0.5,
                    layout=rng.choice(["dense", "fused", "bt"]),
                    ragged=op != "gated_step" and rng.random() < 0.3)
    if op == "clip":
        over = rng.random() < 0.7
        return dict(op=op, sizes="many", n=_log_int(rng, 1, 60), dt=dt, over=over,
                    inplace=not over)
    V, K = _log_int(rng, 50, 128000), rng.choice([0, 1, 2, 4, 7, 12])
    B = max(1, min(_log_int(rng, 1, 64), 16_000_000 // (V * (2 * K + 1))))
    return dict(op=op, B=B, K=K, V=V, dt=dt, q=rng.random() < 0.6, ragged=rng.random() < 0.4,
                temp=rng.choice(["none", "same", "mixed"]))


def _sizes(c):
    """Shapes of the gradients of a clipping case."""
    if c["sizes"] == "layer":
        return [(32, 128), (1, 32, 128), (128,)]
    if c["sizes"] == "model":
        layer = [(1024, 4096), (4, 256, 1024), (4096,)]
        return [(32000, 1024)] + 4 * layer + [(1024, 32000)]
    # any size from one value to two million, the same for every seed
    r = [((i * 2654435761) % 4093) / 4093.0 for i in range(1, c["n"] + 1)]
    return [(int(round(math.exp(x * math.log(2000000.0)))),) for x in r]


# ----------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(shape, dt, g, std=1.0):
    x = torch.randn(shape, generator=g, device=DEV)
    if std != 1.0:
        x.mul_(std)
    return x.to(TYPES[dt])


def _prepare_gated(c, s, g):
    T, B, D, dt = c["T"], c["B"], c["D"], c["dt"]
    # memories from two tokens to several hundred, spread over the channels
    span = torch.exp2(torch.linspace(1.0, 9.0, D, device=DEV))
    if c["gate"] == "logit":
        f = torch.log(span) + torch.randn((T, B, D), generator=g, device=DEV)
    else:
        f = torch.exp(-(0.5 + torch.rand((T, B, D), generator=g, device=DEV)) / span)
    x = torch.randn((T, B, D), generator=g, device=DEV)
    if c["layout"] == "fused":  # halves of one projection
        s["f"], s["x"] = torch.cat([f, x], -1).to(TYPES[dt]).split(D, -1)
    elif c["layout"] == "bt":   # kept batch-first, read time-first
        s["f"], s["x"] = (t.to(TYPES[dt]).transpose(0, 1).contiguous().transpose(0, 1)
                          for t in (f, x))
    else:
        s["f"], s["x"] = f.to(TYPES[dt]), x.to(TYPES[dt])
    s["h0"] = _randn((B, D), "f32", g) if c["state"] else None
    s["lens"] = None
    if c["ragged"]:  # the longest fills the window, the others a half of it or more
        n = torch.randint(T // 2, T + 1, (B,), generator=g, device=DEV)
        n[0] = T
        s["lens"] = n.to(torch.int32)
    if c["op"] == "gated_step":
        s["h1"] = torch.empty((B, D), device=DEV)
    if c["op"] == "gated_bwd":
        s["h"] = _plain_gated(s)["h"]
        s["dh"] = _randn((T, B, D), dt, g, 1e-2)
        s["dhT"] = _randn((B, D), "f32", g, 1e-2) if c["state"] else None


def _prepare_clip(c, s, g):
    s["grads"] = [_randn(n, c["dt"], g, 1e-3) for n in _sizes(c)]
    count = sum(t.numel() for t in s["grads"])
    s["max"] = (0.3 if c["over"] else 30.0) * 1e-3 * math.sqrt(count)
    s["out"] = None if c["inplace"] else [torch.empty_like(t) for t in s["grads"]]


def _prepare_verify(c, s, g):
    B, K, V, dt = c["B"], c["K"], c["V"], c["dt"]
    x = torch.randn((K + 1, B, V), generator=g, device=DEV).mul_(2.0)
    # a few likely continuations for each row, as a trained model has
    hot = torch.randint(0, V, (K + 1, B, 4), generator=g, device=DEV)
    x.scatter_(2, hot, 9.0 + 2.0 * torch.randn((K + 1, B, 4), generator=g, device=DEV))
    s["logits"] = x.to(TYPES[dt])
    t = torch.full((B,), 0.8, device=DEV)
    if c["temp"] == "mixed":  # some of them greedy
        t = 0.5 + torch.rand((B,), generator=g, device=DEV)
        t[::3] = 0.0
    s["temp"] = None if c["temp"] == "none" else t
    s["q"] = None
    if c["q"]:  # the smaller model's view of the same text, its drafts drawn from it
        y = x[:K] + 0.7 * torch.randn((K, B, V), generator=g, device=DEV)
        s["q"] = y.to(TYPES[dt])
        y = s["q"].float() / (1.0 if s["temp"] is None else t[:, None].clamp(min=1e-3))
        u = torch.rand((K, B, V), generator=g, device=DEV).clamp_(min=1e-20)
        s["drafts"] = (y - torch.log(-torch.log(u))).argmax(-1)
    else:
        pick = torch.rand((K, B), generator=g, device=DEV) < 0.7
        s["drafts"] = torch.where(pick, x[:K].argmax(-1), hot[:K, :, 0])
    s["u"] = torch.rand((K + 1, B), generator=g, device=DEV)
    s["n"] = None
    if c["ragged"]:
        s["n"] = torch.randint(0, K + 1, (B,), generator=g, device=DEV).to(torch.int32)


def prepare(case, seed):
    s, g = {"case": dict(case)}, _gen(seed)
    op = case["op"]
    prep = _prepare_clip if op == "clip" else _prepare_verify if op == "verify" else _prepare_gated
    prep(s["case"], s, g)
    return s


# ------------------------------------------------------------ plain forms
def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along the first axis, by doubling: after each
    pass (a, b) spans twice as many steps."""
    d = 1
    while d < a.shape[0]:
        b = torch.cat([b[:d], a[d:] * b[:-d] + b[d:]])
        a = torch.cat([a[:d], a[d:] * a[:-d]])
        d *= 2
    return b


def _gates(s):
    """(keep a, take u, inside a sequence) in float32; outside a keeps all."""
    T, B = s["f"].shape[:2]
    f = s["f"].float()
    if s["case"]["gate"] == "logit":
        a, u = 1.0 / (1.0 + torch.exp(-f)), 1.0 / (1.0 + torch.exp(f))
    else:
        a, u = f, torch.ones_like(f)
    if s["lens"] is None:
        return a, u, None
    live = (torch.arange(T, device=DEV)[:, None] < s["lens"][None, :])[..., None]
    return torch.where(live, a, 1.0), torch.where(live, u, 0.0), live


def _plain_gated(s):
    a, u, live = _gates(s)
    b = u * s["x"].float()
    if s["h0"] is not None:
        b[0] += a[0] * s["h0"]
    h = _scan(a, b)
    last = h[-1].clone()
    if live is not None:
        h = torch.where(live, h, 0.0)
    return {"h": h.to(s["x"].dtype), "hT": last}


def _plain_gated_bwd(s):
    a, u, live = _gates(s)
    x, h = s["x"].float(), s["h"].float()
    dh = s["dh"].float()
    if live is not None:
        dh = torch.where(live, dh, 0.0)
    else:
        dh = dh.clone()
    if s["dhT"] is not None:
        dh[-1] += s["dhT"]
    # backwards in time: g_t = dh_t + a_{t+1} g_{t+1}
    g = _scan(torch.cat([torch.ones_like(a[:1]), a[1:].flip(0)]), dh.flip(0)).flip(0)
    h0 = torch.zeros_like(h[0]) if s["h0"] is None else s["h0"]
    before = torch.cat([h0[None], h[:-1]])
    if s["case"]["gate"] == "logit":
        df = g * (before - x) * a * u
    else:
        df = g * before
    dx = g * u
    if live is not None:
        df, dx = torch.where(live, df, 0.0), torch.where(live, dx, 0.0)
    return {"df": df.to(s["x"].dtype), "dx": dx.to(s["x"].dtype), "dh0": a[0] * g[0]}


def _plain_clip(s):
    total = torch.stack([t.float().square().sum(dtype=torch.float64) for t in s["grads"]]).sum()
    norm = torch.sqrt(total)
    c = torch.where(norm > s["max"], s["max"] / norm, 1.0).float()
    out = s["grads"] if s["out"] is None else s["out"]
    for o, t in zip(out, s["grads"]):
        o.copy_(t.float() * c)
    return {"norm": norm.float(), "grads": out}


def _weights(x, temp):
    """Probabilities of [.., B, V] logits in 64 bits: a border of the cumulated
    sum must not move by the rounding of a hundred thousand terms."""
    x = x.double()
    m = x.amax(-1, keepdim=True)
    if temp is None:
        e = torch.exp(x - m)
        return e / e.sum(-1, keepdim=True)
    t = temp.double()[:, None]
    e = torch.exp((x - m) / torch.where(t > 0, t, 1.0))
    p = e / e.sum(-1, keepdim=True)
    # greedy: all weight on the largest, the lowest index among equals
    V = x.shape[-1]
    at = torch.arange(V, device=x.device)
    first = torch.where(x == m, at, V).amin(-1, keepdim=True)
    return torch.where(t > 0, p, (at == first).double())


def _plain_verify(s):
    c, u = s["case"], s["u"].double()
    K, B, V = c["K"], c["B"], c["V"]
    p = _weights(s["logits"], s["temp"])
    d = s["drafts"].long()
    n = torch.full((B,), K, device=DEV) if s["n"] is None else s["n"].long()
    q = None if s["q"] is None else _weights(s["q"], s["temp"])
    px = p[:K].gather(2, d[..., None])[..., 0]
    qx = torch.ones_like(px) if q is None else q.gather(2, d[..., None])[..., 0]
    k = torch.arange(K, device=DEV)[:, None]
    ok = (u[:K] * qx < px) & (k < n)
    acc = torch.cumprod(ok.long(), 0).sum(0)
    b = torch.arange(B, device=DEV)
    w = p[acc, b]
    if K:
        kk = acc.clamp(max=K - 1)
        if q is None:
            less = torch.zeros_like(w).scatter_(1, d[kk, b][:, None], 1.0)
        else:
            less = q[kk, b]
        r = torch.where((acc < n)[:, None], torch.clamp(w - less, min=0.0), w)
        w = torch.where(r.sum(1, keepdim=True) > 0, r, w)
    cum = torch.cumsum(w, 1)
    new = (cum <= u[K][:, None] * cum[:, -1:]).sum(1)
    # a uniform number at the very end of the sum: the last entry with any weight
    last = torch.where(w > 0, torch.arange(V, device=DEV), 0).amax(1)
    new = torch.minimum(new, last)
    row = torch.arange(K + 1, device=DEV)[:, None]
    full = torch.cat([d, d.new_zeros((1, B))])
    tokens = torch.where(row < acc, full, torch.where(row == acc, new, -1))
    return {"tokens": tokens.int(), "accepted": acc.int()}


def _plain_step(s):
    r = _plain_gated(s)
    return {"h": r["h"], "hT": r["hT"]}


PLAIN = {"gated_fwd": _plain_gated, "gated_step": _plain_step, "gated_bwd": _plain_gated_bwd,
         "clip": _plain_clip, "verify": _plain_verify}


def run(state):
    op = state["case"]["op"]
    return _library(op, state) if own else PLAIN[op](state)


def _library(op, s):
    import gru_recurrence_amd as g
    c = s["case"]
    if op == "gated_fwd":
        h, hT = g.gated_fwd(s["f"], s["x"], s["h0"], gate=c["gate"], lens=s["lens"])
        return {"h": h, "hT": hT}
    if op == "gated_step":
        h, hT = g.gated_step(s["f"], s["x"], s["h0"], gate=c["gate"], h_out=s["h1"])
        return {"h": h, "hT": hT}
    if op == "gated_bwd":
        return g.gated_bwd(s["f"], s["x"], s["h"], s["dh"], s["h0"], s["dhT"], gate=c["gate"],
                           lens=s["lens"])
    if op == "clip":
        norm = g.clip_grads(s["grads"], s["max"], out=s["out"])
        return {"norm": norm, "grads": s["grads"] if s["out"] is None else s["out"]}
    tokens, accepted = g.verify_drafts(s["logits"], s["drafts"], s["u"], s["q"],
                                       temperature=s["temp"], n_drafts=s["n"])
    return {"tokens": tokens, "accepted": accepted}


# ------------------------------------------------------------------- work
def work(case):
    """Each input read once, each output written once."""
    c = case
    e = 2 if c["dt"] == "bf16" else 4
    op = c["op"]
    if op.startswith("gated"):
        n, st = c["T"] * c["B"] * c["D"], c["B"] * c["D"] * 4
        live = 0.75 if c["ragged"] else 1.0  # rows behind a sequence's end are not read
        if op == "gated_bwd":
            return {"bytes": int(4 * n * live + 2 * n) * e + st * (3 if c["state"] else 1),
                    "flops": 10 * n}
        return {"bytes": int(2 * n * live + n) * e + st * (2 if c["state"] else 1), "flops": 6 * n}
    if op == "clip":
        n = sum(math.prod(t) for t in _sizes(c))
        # below the bound in place nothing is written
        return {"bytes": n * e * (1 if c["inplace"] else 2), "flops": 3 * n}
    rows = 1 + c["K"] * (0.5 if c["ragged"] else 1.0) * (2 if c["q"] else 1)
    n = int(c["B"] * rows * c["V"])
    return {"bytes": n * e + c["B"] * (16 * c["K"] + 12), "flops": 5 * n}


# ------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        flat = [t.double() for t in s["grads"]]
        norm = math.sqrt(sum((t * t).sum().item() for t in flat))
        c = s["max"] / norm if norm > s["max"] else 1.0
        return {"norm": torch.tensor(norm, dtype=torch.float64, device=DEV),
                "grads": [t * c for t in flat]}
    return _exact_verify(s) if op == "verify" else _exact_gated(s, op)


def _exact_gated(s, op):
    """Token after token, as the recurrence defines it."""
    T, B, D = s["f"].shape
    logit = s["case"]["gate"] == "logit"
    n = torch.full((B,), T, device=DEV) if s["lens"] is None else s["lens"].long()
    state = torch.zeros((B, D), dtype=torch.float64, device=DEV)
    if s["h0"] is not None:
        state = s["h0"].double()
    if op != "gated_bwd":
        h = torch.zeros((T, B, D), dtype=torch.float64, device=DEV)
        for t in range(T):
            f, x = s["f"][t].double(), s["x"][t].double()
            a = torch.sigmoid(f) if logit else f
            new = a * state + (torch.sigmoid(-f) * x if logit else x)
            if s["lens"] is None:
                state = h[t] = new
            else:
                on = (n > t)[:, None]
                state = torch.where(on, new, state)
                h[t] = torch.where(on, new, 0.0)
        return {"h": h, "hT": state.clone()}
    df, dx = (torch.zeros((T, B, D), dtype=torch.float64, device=DEV) for _ in range(2))
    e = torch.zeros_like(state) if s["dhT"] is None else s["dhT"].double()
    for t in range(T - 1, -1, -1):
        f, x = s["f"][t].double(), s["x"][t].double()
        before = s["h"][t - 1].double() if t else state
        on = (n > t)[:, None]
        g = e + s["dh"][t].double()
        if logit:
            a, u = torch.sigmoid(f), torch.sigmoid(-f)
            dft, dxt = g * (before - x) * a * u, g * u
        else:
            a, dft, dxt = f, g * before, g
        df[t], dx[t] = torch.where(on, dft, 0.0), torch.where(on, dxt, 0.0)
        e = torch.where(on, a * g, e)
    return {"df": df, "dx": dx, "dh0": e}


def _exact_verify(s):
    """Sequence by sequence, draft by draft."""
    c = s["case"]
    K, B, V = c["K"], c["B"], c["V"]
    tokens, accepted = [[-1] * B for _ in range(K + 1)], []
    u, drafts = s["u"].double().cpu(), s["drafts"].cpu()
    temp = None if s["temp"] is None else s["temp"].double().cpu()
    num = None if s["n"] is None else s["n"].cpu()

    def dist(x, b):
        x = x.double()
        if temp is None:
            return torch.softmax(x, -1)
        if temp[b] > 0:
            return torch.softmax(x / temp[b].item(), -1)
        p = torch.zeros_like(x)
        p[int((x == x.max()).nonzero()[0])] = 1.0
        return p
    for b in range(B):
        n, k, less = K if num is None else int(num[b]), 0, None
        while k < n:
            x = int(drafts[k, b])
            p = dist(s["logits"][k, b], b)
            if s["q"] is None:
                q = torch.zeros_like(p)
                q[x] = 1.0
            else:
                q = dist(s["q"][k, b], b)
            if not float(u[k, b]) * float(q[x]) < float(p[x]):
                less = q
                break
            tokens[k][b] = x
            k += 1
        w = p = dist(s["logits"][k, b], b)
        if less is not None:
            w = torch.relu(p - less)
            if not float(w.sum()) > 0:
                w = p
        cum = torch.cumsum(w, 0)
        at = int(torch.searchsorted(cum, (u[K, b].to(DEV) * cum[-1]).reshape(1), right=True))
        tokens[k][b] = min(at, int(w.nonzero()[-1]))
        accepted.append(k)
    return {"tokens": torch.tensor(tokens, dtype=torch.int32, device=DEV),
            "accepted": torch.tensor(accepted, dtype=torch.int32, device=DEV)}
