"""The grouped router's choice in 64 bits, expert by expert, for the tests."""
import numpy as np


def scores(l, kind):
    with np.errstate(all="ignore"):
        if kind == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-l))
        else:
            mx = l.max(1, keepdims=True)
            s = np.exp(l - mx)
            s[np.isneginf(l)] = 0.0
            s = s / s.sum(1, keepdims=True)
    s[np.isneginf(l)] = 0.0
    return s


def choose(l, k, score="sigmoid", bias=None, n_group=1, topk_group=1, group_top=1, renormalize=True, scale=1.0):
    """l [T, E] float64 -> idx [T, k] int32, w [T, k] float64."""
    l = np.asarray(l, np.float64)
    T, E = l.shape
    gs = E // n_group
    b = np.zeros(E) if bias is None else np.asarray(bias, np.float64)
    s = scores(l.copy(), score)
    idx, w = np.zeros((T, k), np.int32), np.zeros((T, k))
    for t in range(T):
        c = s[t] + b
        masked = np.isneginf(b) | np.isneginf(l[t])
        rank = np.where(masked | np.isnan(c), -np.inf, c)
        G = []
        for g in range(n_group):
            best = sorted((v for v in rank[g * gs:(g + 1) * gs] if v != -np.inf), reverse=True)[:group_top]
            G.append(sum(best) if best else -np.inf)
        kept = sorted(range(n_group), key=lambda g: (-G[g], g))[:topk_group]
        cand = [e for g in kept for e in range(g * gs, (g + 1) * gs)]
        idx[t] = sorted(cand, key=lambda e: (-rank[e], e))[:k]
        sv = np.where(np.isneginf(b[idx[t]]), 0.0, s[t][idx[t]])
        if renormalize:
            den = sv.sum()
            sv = np.zeros(k) if den == 0 else sv / den
        w[t] = sv * scale
    return idx, w
