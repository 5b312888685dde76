"""Measured cases of the language-model operators around the recurrence:
the embedding lookup and its gradient, token log probabilities with entropy
and top alternatives and their gradient, and linear attention with a decay
for each head (prompt form, single-token form, backward).

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
        # one decoding step of 16 sequences: ids in, rows out (latency)
        dict(name="embed decode b16", op="embed_fwd", T=1, B=16, V=32000, D=768, dt="bf16",
             ids="i64", order="tb", pad=0.0),
        # a training batch kept batch-first, read in the recurrence's time-first
        # order; vocabulary and ids as a tokenizer gives them
        dict(name="embed prompt t1024 b16", op="embed_fwd", T=1024, B=16, V=50001, D=768,
             dt="bf16", ids="i64", order="bt", pad=0.05),
        # the gradient of that batch, from the float32 dx of the recurrence's backward
        dict(name="embed grad t1024 b16", op="embed_bwd", T=1024, B=16, V=32000, D=768, dt="f32",
             ids="i64", order="bt", pad=0.0),
        # a short ragged batch (a tenth of it padding), odd width, bf16 gradient rows
        dict(name="embed grad ragged", op="embed_bwd", T=301, B=7, V=10007, D=129, dt="bf16",
             ids="i32", order="tb", pad=0.1),
        # sampling step of 16 sequences: chosen token, entropy, 20 alternatives (latency)
        dict(name="logprob decode b16 top20", op="logp_fwd", M=16, V=128000, dt="f32", K=20,
             ids="i64", banned=0.0),
        # scoring of a batch on the projection's float32 logits
        dict(name="logprob score m4096", op="logp_fwd", M=4096, V=32000, dt="f32", K=5,
             ids="i64", banned=0.0),
        # odd vocabulary, bf16 logits, a third of the entries ruled out
        dict(name="logprob ragged banned", op="logp_fwd", M=1001, V=50001, dt="bf16", K=8,
             ids="i32", banned=0.33),
        # gradient of the training loss with an entropy term
        dict(name="logprob grad m4096", op="logp_bwd", M=4096, V=32000, dt="f32", ids="i64",
             banned=0.0),
        # prompt or training forward at the recurrence's headline shape
        dict(name="linattn t1024 b16 nh6", op="lin_fwd", T=1024, B=16, NH=6, NKV=6, Dk=128,
             Dv=128, dt="bf16", state=False, fused=False),
        # one long sequence, few heads, float32 q, k, v as slices of one projection
        dict(name="linattn long f32 nh12", op="lin_fwd", T=8191, B=1, NH=12, NKV=12, Dk=64,
             Dv=64, dt="f32", state=True, fused=True),
        # decoding: 64 sequences, one token each
        dict(name="linattn step b64 nh12", op="lin_step", T=1, B=64, NH=12, NKV=12, Dk=64, Dv=64,
             dt="bf16", state=True, fused=False),
        # training backward, key/value heads shared by two query heads, ragged length
        dict(name="linattn grad t1000 b8", op="lin_bwd", T=1000, B=8, NH=8, NKV=4, Dk=128, Dv=128,
             dt="bf16", state=True, fused=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed_fwd", "embed_bwd", "logp_fwd", "logp_bwd", "lin_fwd", "lin_step",
                     "lin_bwd"])
    dt, ids = rng.choice(["bf16", "f32"]), rng.choice(["i32", "i64"])
    if op.startswith("embed"):
        D = rng.choice([64, 100, 129, 256, 511, 768, 1024])
        T, B = _log_int(rng, 1, 1024), _log_int(rng, 1, 16)
        return dict(op=op, T=T, B=B, V=_log_int(rng, 100, 50000), D=D, dt=dt, ids=ids,
                    order=rng.choice(["tb", "bt"]), pad=rng.choice([0.0, 0.1]))
    if op.startswith("logp"):
        V = _log_int(rng, 50, 128000)
        M = min(_log_int(rng, 1, 4096), max(1, 100_000_000 // V))
        c = dict(op=op, M=M, V=V, dt=dt, ids=ids, banned=rng.choice([0.0, 0.0, 0.33]))
        if op == "logp_fwd":
            c["K"] = min(V, rng.choice([0, 1, 5, 8, 20]))
        return c
    Dk, Dv = rng.choice([32, 48, 64, 96, 128]), rng.choice([32, 64, 80, 128])
    NKV = rng.choice([1, 2, 4, 5, 6])
    NH = NKV * rng.choice([1, 1, 2])
    B = _log_int(rng, 1, 16)
    T = 1 if op == "lin_step" else _log_int(rng, 2, 8191)
    T = max(1, min(T, 100_000 // (B * NH)))
    if op == "lin_step":
        B = _log_int(rng, 1, 128)
    return dict(op=op, T=T, B=B, NH=NH, NKV=NKV, Dk=Dk, Dv=Dv, dt=dt,
                state=op == "lin_step" or rng.random() < 0.5, fused=rng.random() < 0.3)


# ----------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _ids(shape, V, kind, pad, g):
    """Token ids with the skew of text (log-uniform rank); a share `pad` is -1."""
    u = torch.rand(shape, generator=g, device=DEV, dtype=torch.float64)
    t = (torch.exp(u * math.log(V + 1.0)) - 1.0).long().clamp_(0, V - 1)
    if pad:
        t[torch.rand(shape, generator=g, device=DEV) < pad] = -1
    return t.to(torch.int32 if kind == "i32" else torch.int64)


def _randn(shape, dt, g, std=1.0):
    x = torch.randn(shape, generator=g, device=DEV)
    if std != 1.0:
        x.mul_(std)
    return x.to(TYPES[dt])


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    op, dt = c["op"], c["dt"]
    s = {"case": c}
    if op.startswith("embed"):
        T, B, V, D = c["T"], c["B"], c["V"], c["D"]
        bt = c["order"] == "bt"  # kept batch-first, read time-first
        ids = _ids((B, T) if bt else (T, B), V, c["ids"], c["pad"], g)
        s["ids"] = ids.t() if bt else ids
        s["scale"] = math.sqrt(D)
        if op == "embed_fwd":
            s["table"] = _randn((V, D), dt, g, 1.0 / math.sqrt(D))
        else:
            s["dx"] = _randn((T, B, D), dt, g, 1e-2)
    elif op.startswith("logp"):
        M, V = c["M"], c["V"]
        x = torch.randn((M, V), generator=g, device=DEV).mul_(2.0)
        # a few likely continuations for each row, as a trained model has
        hot = torch.randint(0, V, (M, 4), generator=g, device=DEV)
        x.scatter_(1, hot, 6.0 + 3.0 * torch.randn((M, 4), generator=g, device=DEV))
        if c["banned"]:
            x.masked_fill_(torch.rand((V,), generator=g, device=DEV) < c["banned"], -math.inf)
            x[:, hot[0, 0]] = 5.0  # an allowed entry in every row
        s["logits"] = x.to(TYPES[dt])
        del x
        pick = torch.rand((M,), generator=g, device=DEV) < 0.7
        tok = torch.where(pick, hot[:, 0], hot[0, 0])
        s["tok"] = tok.to(torch.int32 if c["ids"] == "i32" else torch.int64)
        if op == "logp_bwd":
            # what a training step has kept from the forward: log-sum-exp and entropy
            s["lse"] = torch.empty((M,), device=DEV)
            s["entropy"] = torch.empty((M,), device=DEV)
            for i in range(0, M, 1024):  # in slices: the double copy stays small
                y = s["logits"][i:i + 1024].double()
                lse = torch.logsumexp(y, 1)
                p = torch.exp(y - lse[:, None])
                s["lse"][i:i + 1024] = lse
                s["entropy"][i:i + 1024] = lse - (p * y.masked_fill(p == 0, 0.0)).sum(1)
            s["dlogp"] = torch.randn((M,), generator=g, device=DEV) * (1.0 / M)
            s["dent"] = torch.randn((M,), generator=g, device=DEV) * (0.01 / M)
    else:
        T, B, NH, NKV, Dk, Dv = (c[k] for k in ("T", "B", "NH", "NKV", "Dk", "Dv"))
        sizes = [NH * Dk, NKV * Dk, NKV * Dv]
        if c["fused"]:  # slices of one projection's output
            x = _randn((T, B, sum(sizes)), dt, g)
            q, k, v = x.split(sizes, -1)
        else:
            q, k, v = (_randn((T, B, n), dt, g) for n in sizes)
        s["q"], s["k"] = q.unflatten(-1, (NH, Dk)), k.unflatten(-1, (NKV, Dk))
        s["v"] = v.unflatten(-1, (NKV, Dv))
        # decays of 1 - 2^-1 .. 1 - 2^-8 spread over the heads
        e = torch.linspace(1.0, 8.0, NH, device=DEV) if NH > 1 else torch.full((1,), 5.0, device=DEV)
        s["g"] = torch.log1p(-torch.exp2(-e))
        s["scale"] = 1.0 / math.sqrt(Dk)
        s["S0"] = _randn((B, NH, Dk, Dv), "f32", g) if c["state"] else None
        if op == "lin_step":
            s["S1"] = torch.empty((B, NH, Dk, Dv), device=DEV)
        if op == "lin_bwd":
            s["do"] = _randn((T, B, NH, Dv), dt, g)
            s["dST"] = _randn((B, NH, Dk, Dv), "f32", g) if c["state"] else None
    return s


# ------------------------------------------------------------ plain forms
def _plain_embed(s):
    ids, table = s["ids"].long(), s["table"]
    ok = ((ids >= 0) & (ids < table.shape[0])).unsqueeze(-1)
    x = table[ids.clamp(0, table.shape[0] - 1)].float() * s["scale"]
    return torch.where(ok, x, 0.0).to(table.dtype)


def _plain_embed_bwd(s):
    V, dx = s["case"]["V"], s["dx"]
    ids = s["ids"].reshape(-1).long()
    rows = dx.reshape(ids.numel(), -1).float() * s["scale"]
    ok = (ids >= 0) & (ids < V)
    out = torch.zeros((V + 1, rows.shape[1]), device=DEV)
    out.index_add_(0, torch.where(ok, ids, V), rows)
    return out[:V]


def _order_key(x):
    """int64 keys in the order (value descending, index ascending) has them, largest first."""
    b = x.view(torch.int32).long()
    b = torch.where(b < 0, -2147483648 - b, b)
    return b * (1 << 20) + ((1 << 20) - 1 - torch.arange(x.shape[1], device=x.device))


def _plain_logp(s):
    x, tok, K = s["logits"].float(), s["tok"].long(), s["case"]["K"]
    m = x.amax(1, keepdim=True)
    z = x - m
    e = torch.exp(z)
    sm = e.sum(1)
    ent = torch.log(sm) - (e * torch.where(e > 0, z, 0.0)).sum(1) / sm
    lse = m[:, 0] + torch.log(sm)
    got = x.gather(1, tok[:, None])[:, 0] - lse
    r = {"logp": got, "entropy": ent, "lse": lse}
    if K:
        key = _order_key(x + 0.0).topk(K, dim=1).values
        top = (1 << 20) - 1 - (key & ((1 << 20) - 1))
        r["top_id"] = top.int()
        r["top_logp"] = x.gather(1, top) - lse[:, None]
    return r


def _plain_logp_bwd(s):
    x, tok = s["logits"].float(), s["tok"].long()
    lp = x - s["lse"][:, None]
    p = torch.exp(lp)
    d = -p * (s["dlogp"][:, None] + s["dent"][:, None] * (torch.where(p > 0, lp, 0.0) + s["entropy"][:, None]))
    d.scatter_add_(1, tok[:, None], s["dlogp"][:, None])
    return d.to(s["logits"].dtype)


def _core(q, k, v, g, X, C=64):
    """o_i = sum_{j<=i} a^(i-j) (q_i k_j) v_j + a^i q_i X and the carried
    X' = a^T X + sum_j a^(T-j) k_j v_j, in chunks of C steps, all chunks at
    once: [B,NH,T,*] in, a = exp(g) for each head."""
    B, NH, T, Dk = q.shape
    n = -(-T // C)
    p = n * C - T
    if p:  # zero rows at the end; the carried state is corrected below
        q, k, v = (torch.cat([t, t.new_zeros((B, NH, p, t.shape[-1]))], 2) for t in (q, k, v))
    q, k, v = (t.reshape(B * NH, n, C, t.shape[-1]) for t in (q, k, v))
    g = g.repeat(B)[:, None, None]
    i = torch.arange(C, device=q.device, dtype=torch.float32)
    lag = i[:, None] - i[None, :]
    D = torch.where(lag >= 0, torch.exp(g * lag.clamp(min=0.0)), 0.0)[:, None]
    o = ((q @ k.transpose(-1, -2)) * D) @ v
    # what each chunk adds to the state carried past it
    w = torch.exp(g * (C - i))[..., None]
    U = (k * w).transpose(-1, -2) @ v
    # carried into chunk c: sum_{c'<c} a^(C (c-1-c')) U_c' + a^(C c) X
    c = torch.arange(n + 1, device=q.device, dtype=torch.float32)
    lag = c[:, None] - 1.0 - c[None, :n]
    W = torch.where(lag >= 0, torch.exp(g * (C * lag.clamp(min=0.0))), 0.0)
    dk, dv = U.shape[-2:]
    S = (W @ U.reshape(B * NH, n, dk * dv)).reshape(B * NH, n + 1, dk, dv)
    if X is not None:
        S = S + torch.exp(g * (C * c))[:, 0, :, None, None] * X.reshape(B * NH, 1, dk, dv)
    o = o + torch.exp(g * i)[:, 0, None, :, None] * (q @ S[:, :n])
    last = S[:, n]
    if p:  # the last chunk holds only C - p rows
        m = C - p
        wl = torch.exp(g * (m - i[:m]))[:, 0, :, None]
        last = torch.exp(g * m) * S[:, n - 1] + (k[:, n - 1, :m] * wl).transpose(-1, -2) @ v[:, n - 1, :m]
    return o.reshape(B, NH, n * C, dv)[:, :, :T], last.reshape(B, NH, dk, dv)


def _bh(t, NH=None):
    """[T,B,h,D] -> float32 [B,NH,T,D], key/value heads repeated for the heads that share them."""
    t = t.float().permute(1, 2, 0, 3)
    return t.repeat_interleave(NH // t.shape[1], 1) if NH else t


def _plain_lin(s):
    q, NH = s["q"], s["q"].shape[2]
    a = torch.exp(s["g"])[:, None, None]
    X = None if s["S0"] is None else a * s["S0"]
    k, v = _bh(s["k"], NH), _bh(s["v"], NH)
    o, last = _core(_bh(q), k, v, s["g"], X)
    # the state after the last token: the carried one before its decay
    T = k.shape[2]
    if T == 1:
        S = k.transpose(-1, -2) @ v if s["S0"] is None else X + k.transpose(-1, -2) @ v
    else:
        S = last / a
    return {"o": (o * s["scale"]).permute(2, 0, 1, 3).to(q.dtype).contiguous(), "S": S}


def _plain_step(s):
    q, k, v = (_bh(s[n], s["q"].shape[2])[:, :, 0] for n in "qkv")
    S = torch.exp(s["g"])[:, None, None] * s["S0"] + k[..., :, None] * v[..., None, :]
    o = (q[..., :, None] * S).sum(-2) * s["scale"]
    return {"o": o[None].to(s["q"].dtype), "S": S}


def _shared(t, NKV):
    """[B,NH,T,D] -> [B,NKV,T,D]: gradients of a shared head added up."""
    B, NH, T, D = t.shape
    return t.reshape(B, NKV, NH // NKV, T, D).sum(2)


def _plain_lin_bwd(s):
    g, NH, NKV, sc = s["g"], s["q"].shape[2], s["k"].shape[2], s["scale"]
    q, k, v, do = _bh(s["q"]), _bh(s["k"], NH), _bh(s["v"], NH), _bh(s["do"])
    a = torch.exp(g)[:, None, None]
    dq, _ = _core(do, v, k, g, None if s["S0"] is None else (a * s["S0"]).transpose(-1, -2))
    qr, kr, vr, dor = (t.flip(2) for t in (q * sc, k, v, do))
    G = s["dST"]
    dv, dS0 = _core(kr, qr, dor, g, G)
    dk, _ = _core(vr, dor, qr, g, None if G is None else G.transpose(-1, -2))
    seq = lambda t: t.permute(2, 0, 1, 3).to(s["q"].dtype).contiguous()  # noqa: E731
    return {"dq": seq(dq * sc), "dk": seq(_shared(dk.flip(2), NKV)),
            "dv": seq(_shared(dv.flip(2), NKV)), "dS0": dS0}


PLAIN = {"embed_fwd": _plain_embed, "embed_bwd": _plain_embed_bwd, "logp_fwd": _plain_logp,
         "logp_bwd": _plain_logp_bwd, "lin_fwd": _plain_lin, "lin_step": _plain_step,
         "lin_bwd": _plain_lin_bwd}


def run(state):
    op = state["case"]["op"]
    return _library(op, state) if own else PLAIN[op](state)


def _library(op, s):
    import gru_recurrence_amd as g
    if op == "embed_fwd":
        return g.embed_fwd(s["ids"], s["table"], s["scale"])
    if op == "embed_bwd":
        return g.embed_bwd(s["ids"], s["dx"], s["case"]["V"], s["scale"])
    if op == "logp_fwd":
        return g.token_logprobs(s["logits"], s["tok"], top=s["case"]["K"])
    if op == "logp_bwd":
        return g.token_logprobs_bwd(s["logits"], s["tok"], s["lse"], s["entropy"], s["dlogp"],
                                    s["dent"])
    if op == "lin_fwd":
        o, S = g.linattn_fwd(s["q"], s["k"], s["v"], s["g"], s["S0"], scale=s["scale"])
        return {"o": o, "S": S}
    if op == "lin_step":
        o, S = g.linattn_step(s["q"], s["k"], s["v"], s["g"], s["S0"], scale=s["scale"],
                              S_out=s["S1"])
        return {"o": o, "S": S}
    return g.linattn_bwd(s["q"], s["k"], s["v"], s["g"], s["do"], s["S0"], s["dST"],
                         scale=s["scale"])


# ------------------------------------------------------------------- work
def work(case):
    """Each input read once, each output written once; products of the
    recurrent form for linear attention."""
    c = case
    e = 2 if c["dt"] == "bf16" else 4
    i = 4 if c.get("ids") == "i32" else 8
    op = c["op"]
    if op.startswith("embed"):
        M = c["T"] * c["B"]
        if op == "embed_fwd":
            # distinct rows of log-uniform ids: sum over ranks of 1 - (1 - p)^M
            return {"bytes": M * i + (_distinct(M, c["V"]) + M) * c["D"] * e, "flops": M * c["D"]}
        return {"bytes": M * i + M * c["D"] * e + c["V"] * c["D"] * 4, "flops": 2 * M * c["D"]}
    if op.startswith("logp"):
        n = c["M"] * c["V"]
        if op == "logp_fwd":
            return {"bytes": n * e + c["M"] * (i + 12 + 8 * c["K"]), "flops": 5 * n}
        return {"bytes": 2 * n * e + c["M"] * (i + 16), "flops": 6 * n}
    n, NH, NKV, Dk, Dv = c["T"] * c["B"], c["NH"], c["NKV"], c["Dk"], c["Dv"]
    state = c["B"] * NH * Dk * Dv * 4
    ins = n * (NH * Dk + NKV * (Dk + Dv)) * e
    if op == "lin_bwd":
        return {"bytes": 2 * ins + n * NH * Dv * e + state * (3 if c["state"] else 1),
                "flops": 10 * n * NH * Dk * Dv}
    return {"bytes": ins + n * NH * Dv * e + state * (2 if c["state"] else 1),
            "flops": 4 * n * NH * Dk * Dv}


def _distinct(M, V):
    L = math.log(V + 1.0)
    n, r = 0.0, 1.0
    while r <= V:  # ranks in groups that grow with the rank
        w = max(1.0, r / 16)
        n += min(w, V + 1 - r) * -math.expm1(M * math.log1p(-min(1.0 - 1e-12, math.log1p(1.0 / r) / L)))
        r += w
    return int(min(M, V, n))


# ------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed_fwd":
        V, D = s["table"].shape
        E = torch.cat([s["table"].double() * s["scale"], s["table"].new_zeros((1, D)).double()])
        ids = s["ids"].long()
        return E.index_select(0, torch.where(ids < 0, V, ids).reshape(-1)).reshape(*ids.shape, D)
    if op == "embed_bwd":
        ids, dx = s["ids"].reshape(-1).long(), s["dx"].double().reshape(-1, s["dx"].shape[-1])
        keep = ids >= 0
        out = torch.zeros((case["V"], dx.shape[1]), dtype=torch.float64, device=DEV)
        out.index_put_((ids[keep],), dx[keep], accumulate=True)
        return out * s["scale"]
    if op == "logp_fwd":
        return _exact_logp(s, case["K"])
    if op == "logp_bwd":
        rows = []
        for i in range(0, case["M"], 512):
            x = s["logits"][i:i + 512].double()
            lp = torch.log_softmax(x, 1)
            p = lp.exp()
            plp = torch.where(p > 0, p * lp, 0.0)
            H = -plp.sum(1, keepdim=True)
            hit = torch.arange(x.shape[1], device=DEV) == s["tok"][i:i + 512].long()[:, None]
            d = s["dlogp"][i:i + 512].double()[:, None] * (hit.double() - p)
            d = d - s["dent"][i:i + 512].double()[:, None] * (plp + p * H)
            rows.append(d)
        return torch.cat(rows)
    return _exact_lin(s, op)


def _exact_logp(s, K):
    out = {"logp": [], "entropy": [], "lse": []}
    if K:
        out["top_logp"], out["top_id"] = [], None
    for x, t in zip(s["logits"].split(512), s["tok"].split(512)):
        x = x.double()
        lp = torch.log_softmax(x, 1)
        out["lse"].append(torch.logsumexp(x, 1))
        out["logp"].append(lp.gather(1, t.long()[:, None])[:, 0])
        out["entropy"].append(torch.special.entr(lp.exp()).sum(1))
        if K:
            out["top_logp"].append(lp.sort(1, descending=True).values[:, :K])
    return {k: torch.cat(v) if v is not None else None for k, v in out.items()}


def _exact_lin(s, op):
    """Token after token, as the recurrence defines it."""
    NH = s["q"].shape[2]
    T, B = s["q"].shape[:2]
    NKV = s["k"].shape[2]
    head = torch.arange(NH, device=DEV) // (NH // NKV)
    q, k, v = s["q"].double(), s["k"].double()[:, :, head], s["v"].double()[:, :, head]
    a = torch.exp(s["g"].double())[None, :, None, None]
    Dk, Dv = q.shape[-1], v.shape[-1]
    S = torch.zeros((B, NH, Dk, Dv), dtype=torch.float64, device=DEV)
    if s["S0"] is not None:
        S = s["S0"].double()
    if op != "lin_bwd":
        o = torch.empty((T, B, NH, Dv), dtype=torch.float64, device=DEV)
        for t in range(T):
            S = a * S + k[t, ..., :, None] * v[t, ..., None, :]
            o[t] = (q[t, ..., None, :] @ S)[..., 0, :] * s["scale"]
        return {"o": o, "S": S}
    do, sc = s["do"].double(), s["scale"]
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    for t in range(T):
        S = a * S + k[t, ..., :, None] * v[t, ..., None, :]
        dq[t] = (S @ do[t, ..., :, None])[..., 0] * sc
    G = torch.zeros_like(S) if s["dST"] is None else s["dST"].double()
    for t in range(T - 1, -1, -1):
        G = G + sc * q[t, ..., :, None] * do[t, ..., None, :]
        dk[t] = (G @ v[t, ..., :, None])[..., 0]
        dv[t] = (k[t, ..., None, :] @ G)[..., 0, :]
        G = a * G
    dk, dv = (torch.zeros((T, B, NKV, t.shape[-1]), dtype=torch.float64, device=DEV).index_add_(2, head, t)
              for t in (dk, dv))
    return {"dq": dq, "dk": dk, "dv": dv, "dS0": G}
