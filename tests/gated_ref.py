"""Plain 64-bit definitions of the gated linear recurrence, of gradient clipping
and of the verification of drafted tokens, on the CPU, for the tests; they share
no code with the library.  The recurrence comes with bounds of what float32
evaluation may be off by.

Its bounds, u = 2^-24 the float32 rounding unit.  The smaller side s of a gate, of
sigmoid(f) and sigmoid(-f), through exponential, sum, reciprocal and product is off
by at most (2 |f| + 6) u relative: the exponent's product and constant |f| u each,
exponential and reciprocal 2 u each, the sum u and the product u.  It is all that is
rounded of the gate: a step is h + s (x - h) or x - s (x - h) and adds the
difference's and its own rounding; time is cut into segments whose products of a and
whose joins add as many roundings again.  With M the recurrence over magnitudes (what
sums and products of either order stay below), the error of h obeys
E_t = a E_{t-1} + u ((2 |f| + 7) s (|x| + M_{t-1}) + 4 M_t), and that of a gradient
through the gate En = a E + u ((2 |f| + 7) s + 4 a) M.  Past |f| = 120 s is 0."""
import numpy as np

U = 2.0 ** -24


def _sig(f):
    """sigmoid(f), sigmoid(-f), both to full relative accuracy."""
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-f)), 1.0 / (1.0 + np.exp(f))


def _lens(lens, T, B):
    n = np.full(B, T) if lens is None else np.clip(np.asarray(lens, np.int64), 0, T)
    return n[:, None]


def gated(f, x, h0, gate, lens=None):
    """Token after token: h, h_T and the bounds of their errors."""
    f, x = np.asarray(f, np.float64), np.asarray(x, np.float64)
    T, B, D = f.shape
    n = _lens(lens, T, B)
    S = np.zeros((B, D)) if h0 is None else np.asarray(h0, np.float64)
    M, E = np.abs(S), np.zeros((B, D))
    h, e = np.zeros((T, B, D)), np.zeros((T, B, D))
    for t in range(T):
        if gate == "logit":
            a, s = _sig(f[t])
            new = a * S + s * x[t]
            m = a * M + s * np.abs(x[t])
            err = a * E + U * ((2 * np.minimum(np.abs(f[t]), 120) + 7) * np.minimum(a, s) * (np.abs(x[t]) + M) + 4 * m)
        else:
            a = np.abs(f[t])
            new = f[t] * S + x[t]
            m = a * M + np.abs(x[t])
            err = a * E + U * 4 * m
        on = n > t
        S, M, E = np.where(on, new, S), np.where(on, m, M), np.where(on, err, E)
        h[t], e[t] = np.where(on, S, 0.0), np.where(on, E, 0.0)
    return h, S, e, E


def gated_grad(f, x, h, dh, h0, dhT, gate, lens=None):
    """df, dx, dh0 and the bounds of their errors, as two dicts."""
    f, h, dh = (np.asarray(t, np.float64) for t in (f, h, dh))
    T, B, D = f.shape
    x = np.zeros_like(f) if x is None else np.asarray(x, np.float64)
    n = _lens(lens, T, B)
    e = np.zeros((B, D)) if dhT is None else np.asarray(dhT, np.float64)
    first = np.zeros((B, D)) if h0 is None else np.asarray(h0, np.float64)
    m, E = np.abs(e), np.zeros((B, D))
    r = {k: np.zeros((T, B, D)) for k in ("df", "dx")}
    b = {k: np.zeros((T, B, D)) for k in ("df", "dx")}
    for t in range(T - 1, -1, -1):
        before = h[t - 1] if t else first
        on = n > t
        g, mg, Eg = e + dh[t], m + np.abs(dh[t]), E
        Eg = Eg + U * mg
        if gate == "logit":
            a, s = _sig(f[t])
            af = np.minimum(np.abs(f[t]), 120)
            df, dx, en = g * (before - x[t]) * a * s, s * g, a * g
            bx = s * (Eg + U * (2 * af + 8) * mg)
            bf = a * s * (np.abs(before) + np.abs(x[t])) * (Eg + U * (4 * af + 16) * mg)
            En = a * Eg + U * ((2 * af + 7) * np.minimum(a, s) + 4 * a) * mg
        else:
            a = np.abs(f[t])
            df, dx, en = g * before, g, f[t] * g
            bx, bf = Eg, np.abs(before) * (Eg + U * mg)
            En = a * Eg + U * 4 * a * mg
        for k, v, w in (("df", df, bf), ("dx", dx, bx)):
            r[k][t], b[k][t] = np.where(on, v, 0.0), np.where(on, w, 0.0)
        e, E, m = np.where(on, en, e), np.where(on, En, E), np.where(on, a * mg, m)
    r["dh0"], b["dh0"] = e, E
    return r, b


def clip(grads, max_norm):
    """(norm, scaled gradients)."""
    g = [np.asarray(t, np.float64) for t in grads]
    norm = np.sqrt(sum((t * t).sum() for t in g))
    c = max_norm / norm if np.isfinite(norm) and norm > max_norm else 1.0
    return norm, [t * c for t in g]


def _dist(x, temp):
    """Probabilities of one row; None where it has none (a NaN, +inf)."""
    if np.isnan(x).any() or (x == np.inf).any():
        return None
    p, m = np.zeros_like(x), x.max()
    if m == -np.inf:
        return p
    if not temp > 0:
        p[int(np.argmax(x))] = 1.0
        return p
    with np.errstate(invalid="ignore"):
        z = np.where(x == -np.inf, -np.inf, (x - m) / temp)
    e = np.exp(z)
    return e / e.sum()


def _draw(w, u):
    if not w.sum() > 0:
        return -1
    cum = np.cumsum(w)
    at = int(np.searchsorted(cum, u * cum[-1], side="right"))
    return min(at, int(np.nonzero(w)[0][-1]))


def verify(logits, drafts, u, q_logits=None, temp=None, n_drafts=None):
    """Sequence after sequence: tokens [K+1,B], accepted [B]."""
    logits = np.asarray(logits, np.float64)
    K, B, V = logits.shape[0] - 1, logits.shape[1], logits.shape[2]
    u = np.clip(np.nan_to_num(np.asarray(u, np.float64), nan=0.0), 0.0, 1.0)
    tokens, accepted = np.full((K + 1, B), -1), np.zeros(B, np.int64)
    for b in range(B):
        n = K if n_drafts is None else int(np.clip(n_drafts[b], 0, K))
        T = 1.0 if temp is None else float(temp[b])
        k, less = 0, np.zeros(V)
        while k < n:
            x, p = int(drafts[k, b]), _dist(logits[k, b], T)
            inside = 0 <= x < V
            if q_logits is None or not T > 0:
                q = np.zeros(V)
                if inside:
                    q[x] = 1.0
            else:
                q = _dist(np.asarray(q_logits[k, b], np.float64), T)
            greedy = not T > 0
            if p is None or not inside:
                ok = False
            elif greedy:
                ok = p[x] == 1.0
            else:
                ok = q is not None and u[k, b] * q[x] < p[x]
            if not ok:
                less = q
                break
            tokens[k, b] = x
            k += 1
        p = _dist(logits[k, b], T)
        accepted[b] = k
        if p is None or less is None:
            continue
        w = np.maximum(p - less, 0.0) if T > 0 else p
        tokens[k, b] = _draw(w if w.sum() > 0 else p, u[K, b])
    return tokens, accepted
