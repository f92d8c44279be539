"""The gate and its gradient in 64 bits, row by row from the formulas."""
import numpy as np


def scores(l, score):
    l = np.asarray(l, np.float64)
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return 1 / (1 + np.exp(-l))
        m = l.max(1, keepdims=True)
        e = np.exp(l - np.where(np.isneginf(m), 0, m))
        total = e.sum(1, keepdims=True)
        return e / np.where(total == 0, 1, total)


def _ranked(v):
    """Positions by value descending, then index ascending; NaN last."""
    return sorted(range(len(v)), key=lambda i: (np.isnan(v[i]), -v[i] if not np.isnan(v[i]) else 0, i))


def gate(logits, k, score="softmax", bias=None, groups=1, top_groups=0, group_best=1, renormalize=True, scale=1.0):
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    s = scores(l, score)
    v = l if bias is None else s + np.asarray(bias, np.float64)
    idx, w = np.zeros((T, k), np.int32), np.zeros((T, k))
    per = E // groups
    for t in range(T):
        allowed = list(range(E))
        if groups > 1 and 0 < top_groups < groups:
            of = s[t] if bias is None and group_best == 2 else v[t]
            value = [np.sort(of[g * per:(g + 1) * per])[::-1][:group_best].sum() for g in range(groups)]
            kept = set(_ranked(value)[:top_groups])
            allowed = [e for e in allowed if e // per in kept]
        best = [allowed[i] for i in _ranked(v[t][allowed])[:k]]
        idx[t] = best
        z = s[t][best]
        if renormalize and score == "softmax":   # the same quotient, without the common factor
            m = l[t][best].max()
            z = np.exp(l[t][best] - m) if m > -np.inf else np.zeros(k)
        if renormalize:
            z = z / z.sum() if z.sum() > 0 else 0 * z
        w[t] = scale * z
    return idx, w


def gate_backward(logits, idx, dw, score, renormalize, scale, d_scores=None):
    """The gradient, and for each element a bound on the magnitudes that were added up for it."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    s = scores(l, score)
    ds = np.zeros((T, E)) if d_scores is None else np.array(d_scores, np.float64)
    mag = np.abs(ds)
    for t in range(T):
        js = [j for j in range(idx.shape[1]) if 0 <= idx[t, j] < E]
        z = s[t][idx[t, js]]
        q = scale * np.asarray(dw, np.float64)[t, js]
        if renormalize:
            S = z.sum()
            g = (q - (q * z).sum() / S) / S if S > 0 else 0 * q
            size = (np.abs(q) + (np.abs(q) * z).sum() / S) / S if S > 0 else 0 * q
        else:
            g, size = q, np.abs(q)
        np.add.at(ds[t], idx[t, js], g)
        np.add.at(mag[t], idx[t, js], size)
    if score == "sigmoid":
        return ds * s * (1 - s), mag * s * (1 - s)
    return s * (ds - (ds * s).sum(1, keepdims=True)), s * (mag + (mag * s).sum(1, keepdims=True))
