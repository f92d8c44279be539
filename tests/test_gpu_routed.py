"""The layer with a given routing, forward and backward, beside the layer that
routes by itself, against 64 bits, and in a whole training step."""
import pytest

import routing_dispatch_expert_amd as moe
from tests.gpu_util import gpu_available, say

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _gpu():
    assert gpu_available(), "GPU tests need an MI355X; run them with -m gpu on a GPU host"
    moe.lib()


def layer(T, d, f, E, dtype, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *s, std=1.0: (torch.randn(*s, device="cuda", generator=g) * std).to(DT[dtype])  # noqa: E731
    return dict(x=rand(T, d), W_router=rand(E, d, std=2 * d ** -0.5), W=[rand(E, f, d, std=d ** -0.5), rand(E, f, d, std=d ** -0.5),
                rand(E, d, f, std=f ** -0.5)], dout=rand(T, d), residual=rand(T, d))


SIZES = [(1, 64, 32, 4, 2, 2.0), (50, 96, 64, 8, 2, 1.0), (700, 256, 128, 16, 4, 1.25), (3000, 128, 64, 64, 6, 0.8), (900, 128, 128, 130, 3, 2.0)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,f,E,k,cf", SIZES)
def test_as_the_layer_that_routes_by_itself(T, d, f, E, k, cf, dtype):
    say("routed", T, d, f, E, k, cf, dtype)
    b = layer(T, d, f, E, dtype)
    r = moe.forward(b["x"], b["W_router"], *b["W"], k=k, cf=cf, P=2, keep_activations=True)
    a = moe.forward_routed(b["x"], r["topk_idx"], r["topk_w"], *b["W"], cf=cf, P=2, keep_activations=True)
    for n in ("out", "slot", "routed_count", "kept_count", "send_count", "totals"):
        assert torch.equal(a[n], r[n]), n
    plain = moe.forward_routed(b["x"], r["topk_idx"], r["topk_w"], *b["W"], cf=cf, P=2)
    assert torch.equal(plain["slot"], r["slot"]) and (plain["out"] - a["out"]).abs().max() <= 2.0 ** -6 * a["out"].abs().max()
    g = moe.backward(b["x"], b["W_router"], *b["W"], b["dout"], k=k, cf=cf, P=2)
    h = moe.backward_routed(b["x"], r["topk_idx"], r["topk_w"], *b["W"], b["dout"], cf=cf, P=2)
    for n in ("dW_gate", "dW_up", "dW_down"):   # the router has no part in these
        assert torch.equal(g[n], h[n]), n
    s = moe.backward_routed(b["x"], r["topk_idx"], r["topk_w"], *b["W"], b["dout"], cf=cf, P=2, saved=a)
    for n in ("dx", "d_topk_w", "dW_gate", "dW_up", "dW_down"):
        assert torch.equal(s[n], h[n]), n


def reference(b, idx, w, slot, x, W, residual):
    """out in 64 bits, as a graph of x, w, W and residual."""
    E = W[0].shape[0]
    out = residual
    for e in range(E):
        t, j = ((idx == e) & (slot >= 0)).nonzero(as_tuple=True)
        if len(t):
            g, u = x[t] @ W[0][e].T, x[t] @ W[1][e].T
            out = out.index_add(0, t, w[t, j][:, None] * ((g * torch.sigmoid(g) * u) @ W[2][e].T))
    return out


@pytest.mark.parametrize("T,d,f,E,k,cf", [(1, 64, 32, 4, 2, 2.0), (60, 100, 68, 5, 3, 0.7), (300, 128, 96, 8, 2, 1.0)])
def test_against_64_bits(T, d, f, E, k, cf):
    b = layer(T, d, f, E, "f32", seed=T)
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    idx = torch.rand(T, E, device="cuda", generator=g).topk(k, 1).indices.int()
    w = torch.randn(T, k, device="cuda", generator=g)
    if T > 1:
        idx[1] = idx[1, 0]                                   # an expert that a token names twice counts twice
        idx[2, 0], idx[3, 0], idx[4] = -1, E, 1 << 30        # no expert
        w[5, 0] = 0
    r = moe.forward_routed(b["x"], idx, w, *b["W"], cf=cf, residual=b["residual"])
    h = moe.backward_routed(b["x"], idx, w, *b["W"], b["dout"], cf=cf)
    x, w64, res = b["x"].double().requires_grad_(), w.double().requires_grad_(), b["residual"].double()
    W = [m.double().requires_grad_() for m in b["W"]]
    out = reference(b, idx, w64, r["slot"], x, W, res)
    # sums of up to 128 products in a row, five of them one after the other, in fp32: some 2^-24 sqrt(128) each, of norms
    assert (r["out"] - out).norm() <= 1e-5 * (out - res).norm() + 2.0 ** -24 * out.norm()
    grads = torch.autograd.grad((out * b["dout"].double()).sum(), (x, w64, *W))
    for n, want in zip(("dx", "d_topk_w", "dW_gate", "dW_up", "dW_down"), grads):
        got = h[n].double()
        if n == "d_topk_w":   # a weight of 0 leaves no trace in the experts' gradients
            want = torch.where(w == 0, 0.0, want)
        assert (got - want).norm() <= 1e-5 * want.norm(), n
    assert not h["d_topk_w"][r["slot"] < 0].any()


@pytest.mark.parametrize("rule", [dict(score="sigmoid", groups=4, top_groups=2, group_best=2, scale=2.5), dict(renormalize=False)], ids=str)
def test_a_training_step(rule):
    """Norm, router, gate and experts, forward and backward, in fp32 against autograd in 64 bits with the same choice."""
    T, d, f, E, k, cf = 120, 128, 64, 16, 4, 1.0
    b = layer(T, d, f, E, "f32", seed=5)
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    nw, bias = 1 + 0.2 * torch.randn(d, device="cuda", generator=g), 0.02 * torch.randn(E, device="cuda", generator=g)
    n = moe.rmsnorm(b["x"], nw, residual=b["residual"])
    logits = n["y"] @ b["W_router"].T
    c = moe.gate(logits, k, bias=bias, **rule)
    r = moe.forward_routed(n["y"], c["topk_idx"], c["topk_w"], *b["W"], cf=cf, residual=n["h"], keep_activations=True)
    e = moe.backward_routed(n["y"], c["topk_idx"], c["topk_w"], *b["W"], b["dout"], cf=cf, saved=r)
    kw = {m: rule[m] for m in ("score", "renormalize", "scale") if m in rule}
    dl = moe.gate_backward(logits, c["topk_idx"], e["d_topk_w"], **kw)
    back = moe.rmsnorm_backward(e["dx"] + dl @ b["W_router"], n["h"], nw, n["rstd"], dh=b["dout"])
    x, res, w, Wr = (t.double().requires_grad_() for t in (b["x"], b["residual"], nw, b["W_router"]))
    W = [m.double().requires_grad_() for m in b["W"]]
    h = x + res
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-6) * w
    l = y @ Wr.T
    s = torch.sigmoid(l) if rule.get("score") == "sigmoid" else torch.softmax(l, 1)
    p = s.gather(1, c["topk_idx"].long())
    p = rule.get("scale", 1.0) * (p / p.sum(1, keepdim=True) if rule.get("renormalize", True) else p)
    out = reference(b, c["topk_idx"], p, r["slot"], y, W, h)
    assert (r["out"] - out).norm() <= 1e-5 * out.norm()
    grads = torch.autograd.grad((out * b["dout"].double()).sum(), (x, res, w, Wr, *W))
    got = (back["dh"], back["dh"], back["dweight"], dl.T @ n["y"], e["dW_gate"], e["dW_up"], e["dW_down"])
    for a, want in zip(got, grads):
        assert (a - want).norm() <= 2e-5 * want.norm()   # ten sums of up to 128 in a row, 2^-24 sqrt(128) each


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_streams_graphs_and_lent_results(dtype):
    b = layer(200, 128, 64, 8, dtype)
    idx = torch.rand(200, 8, device="cuda").topk(2, 1).indices.int()
    w = torch.rand(200, 2, device="cuda")

    def both(s, stream=None):
        s["f"] = moe.forward_routed(b["x"], idx, w, *b["W"], cf=1.0, residual=b["residual"], keep_activations=True, out=s.get("f"), stream=stream)
        s["b"] = moe.backward_routed(b["x"], idx, w, *b["W"], b["dout"], cf=1.0, saved=s["f"], out=s.get("b"), stream=stream)
        return {(m, n): s[m][n].clone() for m, names in (("f", ("out", "slot", "kept_count")),
                ("b", ("dx", "d_topk_w", "dW_gate", "dW_up", "dW_down"))) for n in names}

    same = lambda a, c: all(torch.equal(a[n], c[n]) for n in a)  # noqa: E731
    want = both({})
    other = torch.cuda.Stream()
    s = {}
    for _ in range(2):
        other.wait_stream(torch.cuda.current_stream())
        s["f"] = moe.forward_routed(b["x"], idx, w, *b["W"], cf=1.0, residual=b["residual"], keep_activations=True, out=s.get("f"), stream=other)
        s["b"] = moe.backward_routed(b["x"], idx, w, *b["W"], b["dout"], cf=1.0, saved=s["f"], out=s.get("b"), stream=other)
        torch.cuda.current_stream().wait_stream(other)
        assert all(torch.equal(s[m][n], want[m, n]) for m, n in want)
    torch.cuda.synchronize()
    s = {}
    both(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.forward_routed(b["x"], idx, w, *b["W"], cf=1.0, residual=b["residual"], keep_activations=True, out=s["f"])
        moe.backward_routed(b["x"], idx, w, *b["W"], b["dout"], cf=1.0, saved=s["f"], out=s["b"])
    for seed in (1, 2, 3):
        o = layer(200, 128, 64, 8, dtype, seed)
        b["x"].copy_(o["x"])
        idx.copy_(torch.rand(200, 8, device="cuda").topk(2, 1).indices)
        want = both({})
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(s[m][n], want[m, n]) for m, n in want)
    with pytest.raises(ValueError):
        moe.backward_routed(b["x"], idx, w, *b["W"], b["dout"], cf=2.0, saved=s["f"])
    with pytest.raises(ValueError):
        moe.forward_routed(b["x"], idx, w, *b["W"], cf=1.0, out=s["f"])
    e = moe.forward_routed(b["x"][:0], idx[:0], w[:0], *b["W"], cf=1.0)
    assert e["out"].shape == (0, 128) and not e["kept_count"].any() and not e["totals"].any()
    e = moe.backward_routed(b["x"][:0], idx[:0], w[:0], *b["W"], b["dout"][:0], cf=1.0)
    assert e["dx"].shape == (0, 128) and not e["dW_gate"].any() and not e["dW_down"].any()
