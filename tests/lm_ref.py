"""Plain 64-bit definitions of the operators around the recurrence, on the
CPU, for the tests; they share no code with the library."""
import numpy as np


def embed(ids, table, scale):
    ids, table = np.asarray(ids), np.asarray(table, np.float64)
    V, D = table.shape
    x = np.zeros((*ids.shape, D))
    ok = (ids >= 0) & (ids < V)
    x[ok] = table[ids[ok]] * scale
    return x


def embed_grad(ids, dx, V, scale):
    ids, dx = np.asarray(ids).reshape(-1), np.asarray(dx, np.float64)
    dx = dx.reshape(ids.size, -1)
    out = np.zeros((V, dx.shape[1]))
    for m, i in enumerate(ids):
        if 0 <= i < V:
            out[i] += dx[m]
    return out * scale


def logprobs(logits, tok, K):
    """Row by row: logp, entropy, lse, top_logp, top_id."""
    x = np.asarray(logits, np.float64)
    M, V = x.shape
    logp, ent, lse = np.zeros(M), np.zeros(M), np.zeros(M)
    tl, ti = np.zeros((M, K)), np.zeros((M, K), np.int64)
    for r in range(M):
        row = x[r]
        order = sorted(range(V), key=lambda i: (-row[i], i))[:K]
        m = row.max()
        if m == -np.inf:
            lse[r], ent[r], lp = -np.inf, 0.0, np.full(V, -np.inf)
        else:
            lse[r] = m + np.log(np.exp(row - m).sum())
            lp = row - lse[r]
            p = np.exp(lp)
            ent[r] = -(p[p > 0] * lp[p > 0]).sum()
        logp[r] = lp[tok[r]] if 0 <= tok[r] < V else 0.0
        ti[r], tl[r] = order, lp[order]
    return dict(logp=logp, entropy=ent, lse=lse, top_logp=tl, top_id=ti)


def logprobs_grad(logits, tok, dlogp, dent):
    x = np.asarray(logits, np.float64)
    out = np.zeros_like(x)
    for r in range(x.shape[0]):
        m = x[r].max()
        if m == -np.inf:
            continue
        lp = x[r] - m - np.log(np.exp(x[r] - m).sum())
        p = np.exp(lp)
        plp = np.where(p > 0, p * np.where(p > 0, lp, 0.0), 0.0)
        H = -plp.sum()
        if 0 <= tok[r] < x.shape[1]:
            out[r] -= dlogp[r] * p
            out[r, tok[r]] += dlogp[r]
        out[r] -= dent[r] * (plp + p * H)
    return out


def _heads(t, NH):
    return np.repeat(t, NH // t.shape[2], axis=2)


def linattn(q, k, v, g, S0, scale):
    """Token after token: o [T,B,NH,Dv], S_T."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    T, B, NH, Dk = q.shape
    k, v = _heads(k, NH), _heads(v, NH)
    a = np.exp(np.asarray(g, np.float64))[None, :, None, None]
    S = np.zeros((B, NH, Dk, v.shape[3])) if S0 is None else np.asarray(S0, np.float64)
    o = np.zeros((T, B, NH, v.shape[3]))
    for t in range(T):
        S = a * S + k[t][..., :, None] * v[t][..., None, :]
        o[t] = scale * np.einsum("bhd,bhdv->bhv", q[t], S)
    return o, S


def linattn_grad(q, k, v, g, S0, do, dST, scale):
    q, k, v, do = (np.asarray(t, np.float64) for t in (q, k, v, do))
    T, B, NH, Dk = q.shape
    NKV = k.shape[2]
    k, v = _heads(k, NH), _heads(v, NH)
    Dv = v.shape[3]
    a = np.exp(np.asarray(g, np.float64))[None, :, None, None]
    S = np.zeros((B, NH, Dk, Dv)) if S0 is None else np.asarray(S0, np.float64)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for t in range(T):
        S = a * S + k[t][..., :, None] * v[t][..., None, :]
        dq[t] = scale * np.einsum("bhdv,bhv->bhd", S, do[t])
    G = np.zeros((B, NH, Dk, Dv)) if dST is None else np.asarray(dST, np.float64)
    for t in range(T - 1, -1, -1):
        G = G + scale * q[t][..., :, None] * do[t][..., None, :]
        dk[t] = np.einsum("bhdv,bhv->bhd", G, v[t])
        dv[t] = np.einsum("bhdv,bhd->bhv", G, k[t])
        G = a * G
    share = lambda x: x.reshape(T, B, NKV, NH // NKV, -1).sum(3)  # noqa: E731
    return dict(dq=dq, dk=share(dk), dv=share(dv), dS0=G)
