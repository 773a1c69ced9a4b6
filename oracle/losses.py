"""The row losses in float64, from their definitions: test infrastructure.

Everything is written per row with explicit sums over the allowed tokens; nothing is shared with the
library's kernels."""
import numpy as np


def _row(x, T, allowed):
    """(p, ln p) of one row's allowed tokens (p 0 and ln p -inf elsewhere); None for a row that allows nothing."""
    x = np.where(np.isnan(x), -np.inf, np.asarray(x, np.float64)) / (T if T > 0 else 1.0)
    if allowed is not None:
        x = np.where(allowed, x, -np.inf)
    m = x.max()
    if m == -np.inf:
        return None
    with np.errstate(invalid="ignore"):
        e = np.exp(x - m)
    lp = x - m - np.log(e.sum())
    return np.exp(lp), lp


def policy_loss(logits, tokens, old, adv, ref=None, weight=None, clip_low=0.2, clip_high=0.2, kl=0.0, ent=0.0,
                T=1.0, allowed=None):
    """dict of loss, row_loss, logprob, entropy and grad (all float64)."""
    x = np.asarray(logits, np.float64)
    B, V = x.shape
    w = np.full(B, 1.0 / B) if weight is None else np.asarray(weight, np.float64)
    T = np.broadcast_to(np.asarray(T, np.float64), (B,))
    out = {k: np.zeros(B) for k in ("row_loss", "logprob", "entropy", "slope")}
    grad = np.zeros((B, V))
    for b in range(B):
        i = int(tokens[b])
        if w[b] == 0 or not 0 <= i < V:
            continue
        Tb = T[b] if T[b] > 0 else 1.0
        r = _row(x[b], Tb, None if allowed is None else allowed[b])
        if r is None or r[1][i] == -np.inf:
            out["logprob"][b] = np.nan if r is None else -np.inf
            continue
        p, lp = r
        A, ratio = float(adv[b]), np.exp(lp[i] - float(old[b]))
        one, two = ratio * A, min(max(ratio, 1.0 - clip_low), 1.0 + clip_high) * A
        loss, c = (0.0, 0.0) if A == 0 else ((-one, -one) if one <= two else (-two, 0.0))
        if ref is not None:
            u = float(ref[b]) - lp[i]
            loss += kl * (np.expm1(u) - u)
            c -= kl * np.expm1(u)
        some = p > 0
        H = -np.sum(p[some] * lp[some])
        loss -= ent * H
        g = -c * p
        g[i] += c
        g[some] += ent * p[some] * (lp[some] + H)
        grad[b] = w[b] / Tb * g
        out["row_loss"][b], out["logprob"][b], out["entropy"][b], out["slope"][b] = loss, lp[i], H, c
    out["loss"] = float(sum(w[b] * out["row_loss"][b] for b in range(B) if w[b] != 0))
    out["grad"] = grad
    return out


def preference_loss(logits, tokens, seq_start, weight=None, ref=None, beta=0.1, smooth=0.0, margin=0.0,
                    average=False, T=1.0):
    """dict of loss, pair_loss, reward, logprob, grad and coef (a row's gradient factor, before 1 / T)."""
    x = np.asarray(logits, np.float64)
    N, V = x.shape
    T = T if T > 0 else 1.0
    w = np.ones(N) if weight is None else np.asarray(weight, np.float64)
    lp, prob, counts = np.zeros(N), {}, np.zeros(N, bool)
    for i in range(N):
        t = int(tokens[i])
        if w[i] == 0 or not 0 <= t < V:
            continue
        r = _row(x[i], T, None)
        if r is None or r[1][t] == -np.inf:
            lp[i] = np.nan if r is None else -np.inf
            continue
        lp[i], prob[i], counts[i] = r[1][t], r[0], True
    S = len(seq_start) - 1
    P = S // 2
    R, scale = np.zeros(S), np.ones(S)
    for s in range(S):
        rows = [i for i in range(int(seq_start[s]), int(seq_start[s + 1])) if counts[i]]
        R[s] = sum(w[i] * (lp[i] - (0.0 if ref is None else float(ref[i]))) for i in rows)
        if average:
            n = sum(w[i] for i in rows)
            scale[s] = 1.0 / n if n else 0.0
            R[s] *= scale[s]
    h = beta * (R[:P] - R[P:]) - margin
    pair = (1.0 - smooth) * np.logaddexp(0.0, -h) + smooth * np.logaddexp(0.0, h)
    dh = -(1.0 - smooth) * np.exp(-np.logaddexp(0.0, h)) + smooth * np.exp(-np.logaddexp(0.0, -h))
    coef, grad = np.zeros(N), np.zeros((N, V))
    for s in range(S):
        for i in range(int(seq_start[s]), int(seq_start[s + 1])):
            if counts[i]:
                coef[i] = (1 if s < P else -1) * dh[s % P] * beta / P * scale[s] * w[i]
                grad[i] = -coef[i] / T * prob[i]
                grad[i, int(tokens[i])] += coef[i] / T
    return {"loss": float(pair.mean()) if P else 0.0, "pair_loss": pair, "reward": beta * R, "logprob": lp,
            "grad": grad, "coef": coef}
