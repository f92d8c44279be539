"""Further operators of a mixture-of-experts layer, as measured: the gate (sigmoid
or softmax scores, a bias for balance, groups of experts, top-k, renormalised
weights) and its gradient; the root-mean-square norm in front of the layer with
the residual's addition and an output in 8 bits, and its gradient; 8-bit weights
(quantiser and way back); and the experts' products with 8-bit rows and weights.

Each case is a dict of sizes. prepare() makes its inputs on the GPU from a
seed; run() makes one pass, in plain torch operations in 32 bits (the gate's
scores, which lie next to each other, in 64), or through the package (`own`
true); exact() computes the same outputs in 64 bits from the definitions; work()
gives the bytes and operations of one pass.

An 8-bit matrix [.., N, K] is held as
  codes [.., N, K] float8_e4m3fn
  scale [.., ceil(K/128), N, 4] uint8: byte b of [s, n] is the exponent, biased by
        127, of the scale of row n's columns 128 s + 32 b .. + 31
A value is code * 2^(byte - 127). The scale of a group is the smallest power of
two with |w| <= 448 scale for all of it, 1 (byte 127) if all are zero.
"""
import math

import torch

own = False

MOST = 448.0        # the largest e4m3 value
MOST_FLOPS = 2.8e12  # of a drawn experts' case
MOST_BYTES = 2.5e9   # of weights in a drawn experts' case
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    gate = dict(op="gate", score="sigmoid", bias=True, groups=8, top_groups=4, group_best=2, renormalize=True, scale=2.5)
    norm = dict(op="norm", dtype="bf16", residual=True, y=True, mx8=True)
    back = dict(op="norm_backward", dtype="bf16", residual=True)
    ex = dict(op="experts", dtype="bf16")
    return [
        # the gate of a DeepSeek-V3-shaped layer for one user's next token
        dict(gate, name="gate 1 token", T=1, E=256, k=8),
        # the same for a prefill batch
        dict(gate, name="gate 8192 tokens", T=8192, E=256, k=8),
        # training: softmax scores as they are, with a balance loss's gradient for all of them
        dict(op="gate_backward", name="gate backward, softmax", T=16384, E=64, k=6, score="softmax", renormalize=False, scale=1.0,
             d_scores=True),
        # one user's next token: residual added, bf16 rows for the router, 8 bits for the experts
        dict(norm, name="norm 1 row", R=1, d=7168),
        # a prefill batch of the same
        dict(norm, name="norm 8192 rows", R=8192, d=7168),
        # training, the residual stream's gradient joined
        dict(back, name="norm backward 8192 rows", R=8192, d=4096),
        # a small fp32 model of ragged width
        dict(back, name="norm backward f32, ragged", dtype="f32", residual=False, R=1003, d=500),
        # laying down one layer's matrix in 8 bits, and reading it back
        dict(op="quantize", name="quantize bf16", dtype="bf16", E=4, N=14336, K=4096),
        # fp32 master weights of ragged sizes
        dict(op="quantize", name="quantize f32, ragged", dtype="f32", E=3, N=1000, K=1424),
        # 8-bit experts of the DeepSeek-V3 shape for one user's next token, nothing dropped
        dict(ex, name="experts 1 token", T=1, d=7168, d_ff=2048, E=256, k=8, cf=32.0),
        # and for 64 users' tokens: nearly every expert is hit
        dict(ex, name="experts 64 tokens", T=64, d=7168, d_ff=2048, E=256, k=8, cf=32.0),
        # Mixtral-shaped prefill with a capacity: large products
        dict(ex, name="experts 4096 tokens, 8 experts", T=4096, d=4096, d_ff=14336, E=8, k=2, cf=1.25),
    ]


def _size(rng, lo, hi, q):
    """A multiple of q, spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / q)) * q))


def draw(rng):
    op = rng.choice(("gate", "gate", "gate_backward", "norm", "norm", "norm_backward", "quantize", "experts", "experts", "experts"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op in ("gate", "gate_backward"):
        E = _size(rng, 4, 512, 4)
        c = dict(op=op, T=_size(rng, 1, 16384, 1), E=E, k=_size(rng, 1, min(E // 2, 8), 1),
                 score=rng.choice(("sigmoid", "softmax")), renormalize=rng.random() < 0.6, scale=rng.choice((1.0, 2.5)))
        c["renormalize"] &= c["k"] > 1   # one weight, renormalised, is 1 whatever the scores are
        if op == "gate_backward":
            return dict(c, d_scores=rng.random() < 0.5)
        groups = rng.choice((1, 2, 4))
        c.update(bias=rng.random() < 0.6, groups=groups, top_groups=max(1, groups // 2), group_best=rng.choice((1, 2)))
        if groups // 2 * (E // groups) < c["k"] or E // groups < 2:
            c.update(groups=1, top_groups=1, group_best=1)
        return c
    if op in ("norm", "norm_backward"):
        d = _size(rng, 64, 8192, 16)
        c = dict(op=op, dtype=dtype, R=_size(rng, 1, min(16384, 8192 * 4096 // d), 1), d=d, residual=rng.random() < 0.6)
        if op == "norm":
            c.update(rng.choice((dict(y=True, mx8=True), dict(y=False, mx8=True), dict(y=True, mx8=False))))
        return c
    if op == "quantize":
        return dict(op=op, dtype=dtype, E=_size(rng, 1, 8, 1), N=_size(rng, 16, 7168, 4), K=_size(rng, 64, 4096, 16))
    E = _size(rng, 4, 256, 4)
    c = dict(op=op, dtype="bf16", T=_size(rng, 1, 4096, 1), d=_size(rng, 128, 7168, 16), d_ff=_size(rng, 64, 8192, 16), E=E,
             k=_size(rng, 1, min(E // 2, 8), 1), cf=rng.choice((1.25, 2.0, 4.0)))
    while 3 * c["d"] * c["d_ff"] * E > MOST_BYTES or 6 * c["T"] * c["k"] * c["d"] * c["d_ff"] * c["cf"] > MOST_FLOPS:
        c["T"], c["d_ff"] = max(1, c["T"] // 2), max(64, c["d_ff"] // 32 * 16)
        if c["d_ff"] == 64:
            c["d"] = max(128, c["d"] // 32 * 16)
    return c


# ------------------------------------------------------------------ inputs

def _normal(gen, shape, std, dtype):
    t = torch.empty(shape, dtype=dtype, device="cuda")
    return t.normal_(0.0, std, generator=gen)


def _stream(gen, R, d, dtype):
    """Rows of a residual stream: some channels are much larger than others."""
    channel = torch.exp(0.7 * torch.randn(d, device="cuda", generator=gen))
    return (_normal(gen, (R, d), 1.0, torch.float32) * channel).to(DT[dtype])


def _mx8_random(gen, lead, N, K, std):
    """Codes spread as a quantised Gaussian's, scales that give values of the given deviation."""
    codes = _normal(gen, (*lead, N, K), 170.0, torch.bfloat16).clamp_(-MOST, MOST).to(torch.float8_e4m3fn)
    e = 127 + math.floor(math.log2(std / 170.0))
    scale = torch.randint(e - 1, e + 2, (*lead, -(-K // 128), N, 4), device="cuda", generator=gen, dtype=torch.uint8)
    return dict(codes=codes, scale=scale)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c, s = case, {"case": case}
    if c["op"] in ("gate", "gate_backward"):
        T, E, k = c["T"], c["E"], c["k"]
        s["logits"] = 1.5 * torch.randn((T, E), device="cuda", generator=gen)
        if c["op"] == "gate":
            s["bias"] = 0.05 * torch.randn(E, device="cuda", generator=gen) if c["bias"] else None
            return s
        s["topk_idx"] = torch.rand((T, E), device="cuda", generator=gen).topk(k, 1).indices.int()
        s["d_topk_w"] = torch.randn((T, k), device="cuda", generator=gen)
        s["d_scores"] = 0.1 * torch.randn((T, E), device="cuda", generator=gen) if c["d_scores"] else None
        return s
    if c["op"] in ("norm", "norm_backward"):
        R, d, dt = c["R"], c["d"], DT[c["dtype"]]
        s["x"] = _stream(gen, R, d, c["dtype"])
        s["weight"] = (1 + 0.2 * torch.randn(d, device="cuda", generator=gen)).to(dt)
        s["residual"] = _stream(gen, R, d, c["dtype"]) if c["residual"] else None
        if c["op"] == "norm_backward":
            s["rstd"] = torch.rsqrt(s["x"].double().square().mean(1) + 1e-6).float()   # as the forward kept it
            s["dy"] = _normal(gen, (R, d), 1.0, dt)
        return s
    if c["op"] == "quantize":
        s["W"] = _normal(gen, (c["E"], c["N"], c["K"]), 1 / math.sqrt(c["K"]), DT[c["dtype"]])
        return s
    T, d, f, E, k = c["T"], c["d"], c["d_ff"], c["E"], c["k"]
    s["x"] = _mx8_random(gen, (), T, d, 1.0)
    s["residual"] = _normal(gen, (T, d), 1.0, DT[c["dtype"]])
    s["topk_idx"] = torch.rand((T, E), device="cuda", generator=gen).topk(k, 1).indices.int()
    s["topk_w"] = torch.softmax(torch.randn((T, k), device="cuda", generator=gen), 1)
    for name, n, m in (("W_gate", f, d), ("W_up", f, d), ("W_down", d, f)):
        s[name] = _mx8_random(gen, (E,), n, m, 1 / math.sqrt(m))
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import routing_dispatch_expert_amd as moe
    c = s["case"]
    if c["op"] == "gate":
        r = moe.gate(s["logits"], c["k"], score=c["score"], bias=s["bias"], groups=c["groups"], top_groups=c["top_groups"],
                     group_best=c["group_best"], renormalize=c["renormalize"], scale=c["scale"], out=s.get("result"))
        s["result"] = r   # the outputs are used again by the next pass, here and below
        return {n: r[n] for n in ("topk_idx", "topk_w")}
    if c["op"] == "gate_backward":
        s["result"] = moe.gate_backward(s["logits"], s["topk_idx"], s["d_topk_w"], score=c["score"],
                                        renormalize=c["renormalize"], scale=c["scale"], d_scores=s["d_scores"],
                                        out=s.get("result"))
        return s["result"]
    if c["op"] == "norm":
        r = moe.rmsnorm(s["x"], s["weight"], eps=1e-6, residual=s["residual"], want_y=c["y"], mx8=c["mx8"],
                        out=s.get("result"))
        s["result"] = r
        out = {n: r[n] for n in ("h", "y", "rstd") if r.get(n) is not None}
        if c["mx8"]:
            out["y8"] = moe.dequantize_mx8(r["y8"], torch.bfloat16)
        return out
    if c["op"] == "norm_backward":
        r = moe.rmsnorm_backward(s["dy"], s["x"], s["weight"], s["rstd"], dh=s["residual"], out=s.get("result"))
        s["result"] = r
        return {n: r[n] for n in ("dh", "dweight")}
    if c["op"] == "quantize":
        return moe.dequantize_mx8(moe.quantize_mx8(s["W"]), s["W"].dtype)
    if "handles" not in s:   # the 8-bit matrices' handles, kept by the program as the matrices are
        s["handles"] = [moe.Mx8(s[n]["codes"], s[n]["scale"]) for n in ("x", "W_gate", "W_up", "W_down")]
    x, W_gate, W_up, W_down = s["handles"]
    r = moe.experts_mx8(x, s["topk_idx"], s["topk_w"], W_gate, W_up, W_down, residual=s["residual"], cf=c["cf"],
                        out=s.get("result"))
    s["result"] = r
    return {n: r[n] for n in ("out", "slot", "kept_count")}


def _run_plain(s):
    c = s["case"]
    if c["op"] == "gate":
        return _plain_gate(s, c)
    if c["op"] == "gate_backward":
        return _plain_gate_backward(s, c)
    if c["op"] == "norm":
        x, h = s["x"].float(), s["x"]
        if s["residual"] is not None:
            h = (x + s["residual"].float()).to(h.dtype)   # the stream is kept in its own type, and the norm is of that
            x = h.float()
        rstd = torch.rsqrt(x.square().mean(1) + 1e-6)
        y = x * rstd[:, None] * s["weight"].float()
        out = {"h": h, "rstd": rstd}
        if c["y"]:
            out["y"] = y.to(h.dtype)
        if c["mx8"]:
            out["y8"] = _fake_mx8(y).to(torch.bfloat16)
        return out
    if c["op"] == "norm_backward":
        x, g = s["x"].float() * s["rstd"][:, None], s["dy"].float()
        a = g * s["weight"].float()
        dh = s["rstd"][:, None] * (a - x * (a * x).mean(1, keepdim=True))
        if s["residual"] is not None:
            dh = dh + s["residual"].float()
        return {"dh": dh.to(s["x"].dtype), "dweight": (g * x).sum(0).to(s["x"].dtype)}
    if c["op"] == "quantize":
        return _fake_mx8(s["W"].float()).to(s["W"].dtype)
    return _plain_experts(s, c)


def _fake_mx8(v):
    """The values that v [.., K] has in 8 bits."""
    K = v.shape[-1]
    p = torch.nn.functional.pad(v, (0, -K % 32)).unflatten(-1, (-1, 32))
    m, e = torch.frexp(p.abs().amax(-1, keepdim=True))   # amax = m 2^e, m in [.5, 1); 448 = .875 2^9
    two = torch.where(m > 0, torch.ldexp(torch.ones_like(m), e - 9 + (m > 0.875).int()), torch.ones_like(m))
    q = (p / two).to(torch.float8_e4m3fn).to(v.dtype)
    return (q * two).flatten(-2)[..., :K]


def _values(q, pick=None):
    """The matrices that 8-bit ones stand for, in 32 bits: all, or those that pick names."""
    codes, scale = (t if pick is None else t[pick] for t in (q["codes"], q["scale"]))
    two = torch.ldexp(torch.ones((), device=codes.device), scale.int() - 127)
    two = two.transpose(-3, -2).flatten(-2).repeat_interleave(32, -1)[..., :codes.shape[-1]]
    return codes.float() * two


def _scores(logits, score):
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-logits))
    e = torch.exp(logits - logits.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_gate(s, c):
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    logits = s["logits"].double()
    score = _scores(logits, c["score"])
    order = logits if s["bias"] is None else score + s["bias"].double()   # without a bias the logits' order is the scores'
    if G > 1:
        best = (order if c["group_best"] == 1 else score if s["bias"] is None else order).reshape(T, G, E // G)
        best = torch.sort(best, dim=2, descending=True).values[:, :, :c["group_best"]].sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        keep = torch.zeros_like(best, dtype=torch.bool).scatter_(1, kept, True)
        order = order.masked_fill(~keep.repeat_interleave(E // G, dim=1), -math.inf)
    idx = torch.sort(order, dim=1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, idx)
    if c["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    return {"topk_idx": idx.int(), "topk_w": (c["scale"] * w).float()}


def _plain_gate_backward(s, c):
    score = _scores(s["logits"], c["score"])
    idx, dw = s["topk_idx"].long(), s["d_topk_w"] * c["scale"]
    if c["renormalize"]:
        w = score.gather(1, idx)
        total = w.sum(1, keepdim=True)
        dw = (dw - (dw * w).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(score) if s["d_scores"] is None else s["d_scores"]
    ds = ds.scatter_add(1, idx, dw)
    if c["score"] == "sigmoid":
        return ds * score * (1 - score)
    return score * (ds - (ds * score).sum(1, keepdim=True))


def _slots(idx, E, C):
    """Rank of each copy among its expert's copies in token order (-1: at or over the capacity), and the counts kept."""
    flat = idx.reshape(-1).long()
    hot = (flat[:, None] == torch.arange(E, device=flat.device)).int()
    rank = (torch.cumsum(hot, 0) * hot).sum(1) - 1
    slot = torch.where(rank < C, rank, torch.full_like(rank, -1)).reshape(idx.shape)
    return slot.int(), hot.sum(0).clamp(max=C).int()


def _capacity(c):
    return math.ceil(float(torch.tensor(c["cf"], dtype=torch.float32)) * c["k"] * c["T"] / c["E"])


def _plain_experts(s, c):
    T, E, k, C = c["T"], c["E"], c["k"], _capacity(c)
    slot, kept = _slots(s["topk_idx"], E, C)
    e, at = s["topk_idx"].reshape(-1).long(), slot.reshape(-1).long()
    rows = _values(s["x"]).repeat_interleave(k, 0)
    if T * k <= E // 2:   # few copies: each one's matrices
        pick, x = e, rows[:, :, None]
    else:   # every expert's rows in a bucket
        fits = torch.where(at >= 0, at, torch.full_like(at, C))
        bucket = torch.zeros((E, C + 1, rows.shape[1]), device=rows.device)
        bucket[e, fits] = rows
        pick, x = None, bucket[:, :C].transpose(1, 2).contiguous()
    g = torch.bmm(_values(s["W_gate"], pick), x)
    h = g / (1 + torch.exp(-g)) * torch.bmm(_values(s["W_up"], pick), x)
    h = _fake_mx8(h.transpose(1, 2)).transpose(1, 2).contiguous()   # the activations between the products are in 8 bits too
    y = torch.bmm(_values(s["W_down"], pick), h).transpose(1, 2)
    y = y[:, 0] if pick is not None else y[e, at.clamp(min=0)]
    part = torch.where((at >= 0)[:, None], s["topk_w"].reshape(-1, 1) * y, torch.zeros_like(y))
    out = s["residual"].float() + part.reshape(T, k, -1).sum(1)
    return {"out": out.to(s["residual"].dtype), "slot": slot, "kept_count": kept}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s, c = prepare(case, seed), case
    return {"gate": _exact_gate, "gate_backward": _exact_gate_backward, "norm": _exact_norm,
            "norm_backward": _exact_norm_backward, "quantize": lambda s, c: _exact_mx8(s["W"].double()),
            "experts": _exact_experts}[c["op"]](s, c)


def _exact_gate(s, c):
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    l = s["logits"].double()
    p = torch.softmax(l, 1) if c["score"] == "softmax" else torch.sigmoid(l)
    value = l if s["bias"] is None else p + s["bias"].double()
    allowed = torch.ones_like(l, dtype=torch.bool)
    if G > 1:
        v = (p if s["bias"] is None and c["group_best"] > 1 else value).reshape(T, G, E // G)
        best = v.topk(c["group_best"], 2).values.sum(2)
        # a group's place: how many groups are better, or as good and before it
        ahead = (best[:, None, :] > best[:, :, None]) | ((best[:, None, :] == best[:, :, None])
                                                         & torch.ones(G, G, device=l.device).tril(-1).bool())
        allowed = (ahead.sum(2) < c["top_groups"])[:, :, None].expand(T, G, E // G).reshape(T, E)
    chosen = []
    for _ in range(k):   # argmax takes the first of equals only where told: the lowest index of the largest value
        top = value.masked_fill(~allowed, -math.inf)
        top = (top == top.amax(1, keepdim=True)) & allowed
        i = torch.where(top, torch.arange(E, device=l.device), E).amin(1, keepdim=True)
        allowed = allowed.scatter(1, i, False)
        chosen.append(i)
    i = torch.cat(chosen, 1)
    w = p.gather(1, i)
    if c["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    return {"topk_idx": i.int(), "topk_w": w * c["scale"]}


def _exact_gate_backward(s, c):
    l = s["logits"].double().requires_grad_()
    p = torch.softmax(l, 1) if c["score"] == "softmax" else torch.sigmoid(l)
    w = p.gather(1, s["topk_idx"].long())
    if c["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    loss = (c["scale"] * w * s["d_topk_w"].double()).sum()
    if s["d_scores"] is not None:
        loss = loss + (p * s["d_scores"].double()).sum()
    return torch.autograd.grad(loss, l)[0]


def _exact_mx8(v):
    """Of v in 64 bits: the values nearest to it on the grid of its group's scale, halfway to the even mantissa."""
    K = v.shape[-1]
    p = torch.nn.functional.pad(v, (0, -K % 32)).unflatten(-1, (-1, 32))
    big = p.abs().amax(-1, keepdim=True)
    two = torch.exp2(torch.ceil(torch.log2(torch.where(big > 0, big, torch.full_like(big, MOST)) / MOST)))
    two = torch.where(big > MOST * two, two * 2, torch.where(big <= MOST * two / 2, two / 2, two))   # the logarithm's own rounding
    r = p / two
    step = torch.exp2(torch.floor(torch.log2(r.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(r / step) * step * two).flatten(-2)[..., :K]


def _exact_norm(s, c):
    h = s["x"]
    if s["residual"] is not None:
        h = (h.double() + s["residual"].double()).to(h.dtype)   # kept in its own type by definition
    v = h.double()
    rstd = 1 / torch.sqrt((v * v).sum(1) / c["d"] + 1e-6)
    y = v * rstd[:, None] * s["weight"].double()
    out = {"h": h.double(), "rstd": rstd}
    if c["y"]:
        out["y"] = y
    if c["mx8"]:
        out["y8"] = _exact_mx8(y)
    return out


def _exact_norm_backward(s, c):
    h, r, w, dy = (s[n].double() for n in ("x", "rstd", "weight", "dy"))
    n = h * r[:, None]
    dot = (dy * w * n).sum(1) / c["d"]
    dh = (dy * w - n * dot[:, None]) * r[:, None]
    if s["residual"] is not None:
        dh = dh + s["residual"].double()
    return {"dh": dh, "dweight": (dy * n).sum(0)}


def _exact_matrix(q, e=None):
    codes, scale = (t if e is None else t[e] for t in (q["codes"], q["scale"]))
    N, K = codes.shape
    k = torch.arange(K, device=codes.device)
    byte = scale[k // 128, :, k // 32 % 4].T   # [N, K]
    return codes.double() * torch.exp2(byte.double() - 127)


def _exact_experts(s, c):
    T, E, k, C = c["T"], c["E"], c["k"], _capacity(c)
    copies, slots = [[] for _ in range(E)], []
    for t, mine in enumerate(s["topk_idx"].tolist()):
        for j, e in enumerate(mine):
            slots.append(len(copies[e]) if len(copies[e]) < C else -1)
            if len(copies[e]) < C:
                copies[e].append((t, j))
    x, w = _exact_matrix(s["x"]), s["topk_w"].double()
    out = s["residual"].double()
    for e, mine in enumerate(copies):
        if not mine:
            continue
        t, j = torch.tensor(mine, device=x.device).T
        g = x[t] @ _exact_matrix(s["W_gate"], e).T
        h = _exact_mx8(g * torch.sigmoid(g) * (x[t] @ _exact_matrix(s["W_up"], e).T))
        out.index_add_(0, t, w[t, j][:, None] * (h @ _exact_matrix(s["W_down"], e).T))
    dev = x.device
    return {"out": out, "slot": torch.tensor(slots, dtype=torch.int32, device=dev).reshape(T, k),
            "kept_count": torch.tensor([len(m) for m in copies], dtype=torch.int32, device=dev)}


# ------------------------------------------------------------------ work

def work(case):
    c = case
    eb = 2 if c.get("dtype") == "bf16" else 4
    q8 = 1 + 1 / 32
    if c["op"] == "gate":   # scores of about ten operations each, compared with log2(k) + 1 others
        return {"bytes": c["T"] * (c["E"] * 4 + c["k"] * 8), "flops": 12 * c["T"] * c["E"]}
    if c["op"] == "gate_backward":
        return {"bytes": c["T"] * (c["E"] * 4 * (2 + c["d_scores"]) + c["k"] * 8), "flops": 12 * c["T"] * c["E"]}
    if c["op"] == "norm":
        n = c["R"] * c["d"]
        return {"bytes": n * (eb * (1 + 2 * c["residual"] + c["y"]) + c["mx8"] * q8) + c["d"] * eb + 4 * c["R"], "flops": 8 * n}
    if c["op"] == "norm_backward":
        n = c["R"] * c["d"]
        return {"bytes": n * eb * (3 + c["residual"]) + 2 * c["d"] * eb + 4 * c["R"], "flops": 12 * n}
    if c["op"] == "quantize":   # weights in, codes out; codes in, weights out
        n = c["E"] * c["N"] * c["K"]
        return {"bytes": n * (2 * eb + 2 * q8), "flops": 4 * n}
    T, d, f, E, k = c["T"], c["d"], c["d_ff"], c["E"], c["k"]
    hit = E * (1 - (1 - k / E) ** T)              # distinct experts, as uniform routing gives them
    copies = min(T * k, E * _capacity(c))
    return {"bytes": hit * 3 * d * f * q8 + T * d * (q8 + 2 * eb) + 8 * T * k, "flops": 6 * copies * d * f}
