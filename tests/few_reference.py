"""The few-token layer and the 4-bit weights in 64 bits, from the definitions
in include/moe.h, with the bounds that their outputs have to keep. Shares no
code with the kernels; the routing comes from the oracle."""
from __future__ import annotations

import math

import numpy as np

import moe_inputs
import oracle

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])
STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}   # largest relative error of one rounding to nearest
# One step of an fp32 sum or product, taken as 2^-23 (twice the error of a
# rounding to nearest): the matrix instructions' inner sums may cut off.
ACC = 2.0 ** -23


def q4_shapes(E, N, K, group):
    nt, kt = -(-N // 16), -(-K // 128)
    return (E, nt, kt, 1024), (E, nt, kt * (128 // group), 16)


def q4_locate(N, K, kind):
    """Index of tile, byte and half of every weight [N, K] of one matrix."""
    n, k = np.arange(N)[:, None], np.arange(K)[None, :]
    i = k % 8
    bit = np.where(i % 2 == 0, 2 * i, 14 + 2 * i) if kind == "u4" else 4 * i
    byte = 16 * (16 * (k % 32 // 8) + n % 16) + 4 * (k % 128 // 32) + bit // 8
    return n // 16 + 0 * k, k // 128 + 0 * n, byte, bit % 8 // 4 + 0 * n


def q4_decode(codes, scale64, zero, shape, group, kind):
    """(W, |W| as the sums' error bound sees it), [E, N, K] float64. A u4 weight
    enters the sums as s (16 + q) and s (16 + z), whose magnitudes add."""
    E, N, K = shape
    tn, tk, byte, half = q4_locate(N, K, kind)
    q = (codes[:, tn, tk, byte] >> (4 * half).astype(np.uint8)) & 15
    g = np.arange(K)[None, :] // group + 0 * tn
    r = np.arange(N)[:, None] % 16 + 0 * g
    s = scale64[:, tn, g, r]
    if kind == "u4":
        z = np.full(s.shape, 8.0) if zero is None else zero[:, tn, g, r].astype(np.float64)
        return s * (q.astype(np.float64) - z), np.abs(s) * (32 + q + z)
    return s * E2M1[q], np.abs(s * E2M1[q])


def q4_quantize(W32, group, kind, zero_points):
    """codes (padding 0 standing for zero weights), scale (float32 values), zero of fp32 weights [E, N, K]."""
    E, N, K = W32.shape
    f = np.float32
    (_, nt, kt, _), sshape = q4_shapes(E, N, K, group)
    w = np.zeros((E, nt * 16, kt * 128), f)
    w[:, :N, :K] = W32
    w = w.reshape(E, nt * 16, -1, group)
    lo, hi = np.minimum(w.min(-1), f(0)), np.maximum(w.max(-1), f(0))
    big = np.maximum(hi, -lo)
    span = big * (f(1) / f(6)) if kind == "e2m1" else (hi - lo) * (f(1) / f(15)) if zero_points else big * (f(1) / f(7))
    s = moe_inputs.bits_to_f64(moe_inputs.to_bf16_bits(span), "bf16").astype(f)
    one = np.where(s > 0, s, f(1))
    r = (w / one[..., None]).astype(f)
    z = np.zeros(s.shape, f)
    if kind == "e2m1":
        d = np.abs(np.abs(r.astype(np.float64))[..., None] - E2M1[:8])
        near = d == d.min(-1, keepdims=True)
        first, last = near.argmax(-1), 7 - near[..., ::-1].argmax(-1)   # differ where two are equally near
        q = np.where(first % 2 == 0, first, last) + np.where(r < 0, 8, 0)
    elif zero_points:
        z = np.where(s > 0, np.clip(np.rint(-lo / one), 0, 15), 0).astype(f)
        q = np.where(s[..., None] > 0, np.clip(np.rint(r) + z[..., None], 0, 15), 0)
    else:
        z += 8
        q = np.clip(np.rint(r) + 8, 0, 15)
    q = np.where(s[..., None] > 0, q, 0 if kind == "e2m1" or zero_points else 8)
    q = q.reshape(E, nt * 16, -1).astype(np.uint8)
    tn, tk, byte, half = q4_locate(nt * 16, kt * 128, kind)
    codes = np.zeros((E, nt, kt, 1024), np.uint8)
    for h in (0, 1):
        m = half == h
        np.bitwise_or.at(codes, (slice(None), tn[m], tk[m], byte[m]), (q[:, m] << (4 * h)).astype(np.uint8))
    tiled = [t.reshape(E, nt, 16, -1).transpose(0, 1, 3, 2).copy() for t in (s, z.astype(np.uint8))]
    return codes, tiled[0], tiled[1] if kind == "u4" and zero_points else None


def random_q4(rng, E, N, K, group, kind, zero_points):
    """Random codes, scales as bf16 bits and zero points: every byte of the layout is drawn, padding too."""
    cs, ss = q4_shapes(E, N, K, group)
    codes = rng.integers(0, 256, cs, dtype=np.uint8)
    scale = moe_inputs.to_bf16_bits((0.5 + rng.random(ss, dtype=np.float32)) / (4.6 * math.sqrt(K)))
    zero = rng.integers(0, 16, ss, dtype=np.uint8) if kind == "u4" and zero_points else None
    return codes, scale, zero


def routing(wl):
    """The layer's routing of a generated workload, from the oracle, with gates in 64 bits."""
    x, wr = oracle.decode(wl.x, wl.dtype), oracle.decode(wl.wr, wl.dtype)
    bias = None if wl.bias_vec is None else wl.bias_vec.astype(np.float64)
    logits = x @ wr.T + (0 if bias is None else bias)
    if 0 < wl.max_ranks < wl.P:
        idx = oracle.rank_limited_experts(logits, wl.k, wl.P, wl.max_ranks)
    else:
        idx = oracle.topk_experts(logits, wl.k)
    top = np.take_along_axis(logits, idx.astype(np.int64), 1)
    w = np.exp(top - top[:, :1])
    w /= w.sum(1, keepdims=True)
    C = oracle.capacity(wl.T, wl.E, wl.k, wl.cf)
    count, slot = np.zeros(wl.E, np.int32), np.full(idx.shape, -1, np.int32)
    for t in range(wl.T):
        for j in range(wl.k):
            e = idx[t, j]
            slot[t, j] = count[e] if count[e] < C else -1
            count[e] += 1
    kept = np.minimum(count, C)
    send = kept.reshape(wl.P, -1).sum(1)
    totals = [int(wl.T * wl.k - kept.sum()), int((slot < 0).all(1).sum()), int(wl.E * C - kept.sum()),
              int((kept.sum() - send[0]) * wl.d * wl.elem_bytes)]
    # a score: pieces of at most 32 products in fp32, added up in fp64; a gate's relative error is twice a score's
    mag = (np.abs(x) @ np.abs(wr).T).max()
    return dict(x=x, idx=idx, w=w, w_err=2 * 33 * ACC * mag + 2.0 ** -23, slot=slot, routed=count, kept=kept, send=send,
                totals=totals, C=C)


def layer(wl, weights, r):
    """(out, bound) in 64 bits. weights: name -> e -> (W, |W|) as q4_decode gives them.

    Sums of n terms in fp32 are off by at most n ACC times the sum of the
    magnitudes. For h: |silu'| <= 1.1 and |silu(g)| <= |g|, and the rounding of
    h to the layer's type. The combine adds k + 1 terms, and out is rounded
    once. Errors of second order are covered by the factor 1.01."""
    step = STEP[wl.dtype]
    out, err = r["x"].copy(), np.zeros_like(r["x"])
    nd, nf = wl.d + 8, wl.d_ff + 8
    for e in np.nonzero(r["kept"])[0]:
        at = [(t, j) for t in range(wl.T) for j in range(wl.k) if r["idx"][t, j] == e and r["slot"][t, j] >= 0]
        t = [a for a, _ in at]
        w = np.array([r["w"][a] for a in at])[:, None]
        X, (Wg, Ag), (Wu, Au), (Wd, Ad) = r["x"][t], weights["g"](e), weights["u"](e), weights["d"](e)
        g, u = X @ Wg.T, X @ Wu.T
        eg, eu = nd * ACC * (np.abs(X) @ Ag.T), nd * ACC * (np.abs(X) @ Au.T)
        sg = g / (1 + np.exp(-g))
        h = sg * u
        # the exponential and the quotient: 8 steps of fp32 on top
        eh = 1.01 * (1.1 * eg * np.abs(u) + (np.abs(sg) + 1.1 * eg) * eu) + (step + 8 * ACC) * np.abs(h)
        y = h @ Wd.T
        ey = eh @ np.abs(Wd).T + nf * ACC * ((np.abs(h) + eh) @ Ad.T)
        np.add.at(out, t, w * y)
        np.add.at(err, t, 1.01 * w * ey + (r["w_err"] + (wl.k + 2) * ACC) * w * np.abs(y))
    return out, 1.01 * err + (step + (wl.k + 1) * ACC) * np.abs(out) + 1e-30
