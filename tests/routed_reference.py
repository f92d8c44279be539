"""The gradients of the layer with a given routing in 64 bits, with a bound on each element's error.

The kernels store X, g, u, h, dy, dh, dg, du and dX in the layer's type (each rounded by half a step, `half` of itself, or
near zero by less than 2^-126), and sum in fp32 (each addition and product off by 2^-23 of the magnitudes: the matrix
instructions may cut off). The bounds below carry these through the formulas, product by product."""
import torch

U = 2.0 ** -24
TINY = 2.0 ** -126


def _times(a, ea, b, eb):
    """The error of a b."""
    return a.abs() * eb + ea * b.abs() + ea * eb


def gradients(x, idx, w, slot, W, dout, half):
    """{name: (value, bound)} of dx, d_topk_w, dW_gate, dW_up, dW_down; "parts" [T]: the norms of the copies' parts of dx,
    added in squares; "terms" [T, k]: the terms of d_topk_w, the same. Tensors of 64 bits; idx and slot as they are."""
    T, k = idx.shape
    d, F, E = x.shape[1], W[0].shape[1], W[0].shape[0]
    dx, edx, size = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    dw, edw, terms, parts = torch.zeros_like(w), torch.zeros_like(w), torch.zeros_like(w), torch.zeros_like(w[:, 0])
    dW, eW = [torch.zeros_like(m) for m in W], [torch.zeros_like(m) for m in W]
    stored = lambda v, e, times=1: e + times * half * (v.abs() + e) + TINY  # noqa: E731
    for e in range(E):
        t, j = ((idx == e) & (slot >= 0)).nonzero(as_tuple=True)
        n = len(t)
        if not n:
            continue
        X, Wg, Wu, Wd, weight = x[t], W[0][e], W[1][e], W[2][e], w[t, j][:, None]
        g, u = X @ Wg.T, X @ Wu.T
        eg, eu = (stored(v, 2 * U * d * (X.abs() @ m.abs().T)) for v, m in ((g, Wg), (u, Wu)))
        s = torch.sigmoid(g)
        slope = s * (1 + g * (1 - s))
        # silu' is at most 1.1 and changes by at most 1/2; the exponential, sums and quotient: eight roundings
        silu, esilu, eslope = g * s, 1.1 * eg + 8 * U * (g * s).abs(), 0.5 * eg + 9 * U
        h = silu * u
        eh = stored(h, _times(silu, esilu, u, eu) + 2 * U * h.abs())
        # dout as dy for a weight of 1: what the weight does to dy and dh, it does to their errors (dh is rounded twice at most)
        dy = dout[t]
        dh = dy @ Wd
        edy = stored(dy, 0 * dy)
        edh = stored(dh, edy @ Wd.abs() + 2 * U * d * (dy.abs() @ Wd.abs()), 2)
        dw[t, j] = (dh * h).sum(1)
        terms[t, j] = (dh * h).norm(dim=1)
        edw[t, j] = (_times(dh, edh, h, eh) + 2 * U * F * (dh * h).abs()).sum(1) + 2 * U * (dh * h).sum(1).abs()
        dy, edy, dh, edh = weight * dy, weight.abs() * edy + TINY, weight * dh, weight.abs() * edh + TINY
        a, ea = u * slope, _times(u, eu, slope, eslope)
        dg, du = dh * a, dh * silu
        edg = stored(dg, _times(dh, edh, a, ea) + 4 * U * dg.abs())
        edu = stored(du, _times(dh, edh, silu, esilu) + 4 * U * du.abs())
        part = dg @ Wg + du @ Wu
        mag = dg.abs() @ Wg.abs() + du.abs() @ Wu.abs()
        epart = stored(part, edg @ Wg.abs() + edu @ Wu.abs() + 4 * U * F * mag)
        dx.index_add_(0, t, part)
        edx.index_add_(0, t, epart)
        size.index_add_(0, t, part.abs() + epart)
        parts.index_add_(0, t, part.square().sum(1))
        for i, (l, el, r, er) in enumerate(((dg, edg, X, 0 * X), (du, edu, X, 0 * X), (dy, edy, h, eh))):
            dW[i][e] = l.T @ r
            err = l.abs().T @ er + el.T @ r.abs() + el.T @ er + 2 * U * n * ((l.abs() + el).T @ (r.abs() + er))
            eW[i][e] = stored(dW[i][e], err)
    edx = stored(dx, edx + k * U * size)
    return {"dx": (dx, edx), "d_topk_w": (dw, edw), "dW_gate": (dW[0], eW[0]), "dW_up": (dW[1], eW[1]), "dW_down": (dW[2], eW[2]),
            "parts": parts.sqrt(), "terms": terms}
