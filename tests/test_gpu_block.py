"""The norm, the gate and the 8-bit experts together, as a transformer block
uses them: the whole layer, a training step through norm and gate, other streams,
captured calls, and lent results."""
import numpy as np
import pytest

import routing_dispatch_expert_amd as moe
from tests.gpu_util import gpu_available, say

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
RULES = [dict(score="sigmoid", groups=4, top_groups=2, group_best=2, scale=2.5), dict(renormalize=False), dict(score="sigmoid", renormalize=False),
         dict(groups=4, top_groups=3)]


@pytest.fixture(autouse=True)
def _gpu():
    assert gpu_available(), "GPU tests need an MI355X; run them with -m gpu on a GPU host"
    moe.lib()


def block(T, d, f, E, dtype="bf16", seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *s, std=1.0: (torch.randn(*s, device="cuda", generator=g) * std).to(DT[dtype])  # noqa: E731
    full = [rand(E, f, d, std=d ** -0.5), rand(E, f, d, std=d ** -0.5), rand(E, d, f, std=f ** -0.5)]
    return dict(x=rand(T, d), norm_weight=1 + 0.2 * rand(d), W_router=rand(E, d, std=2 * d ** -0.5),
                W=[moe.quantize_mx8(w) for w in full], residual=rand(T, d), bias=0.02 * torch.randn(E, device="cuda", generator=g))


def call(b, k, cf, residual=True, bias=True, **kw):
    return moe.forward_mx8(b["x"], b["norm_weight"], b["W_router"], *b["W"], k, cf, residual=b["residual"] if residual else None,
                           bias=b["bias"] if bias else None, **kw)


def same(a, b, names=("out", "h", "y", "logits", "topk_idx", "topk_w", "slot", "routed_count", "kept_count")):
    for n in names:
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rule", RULES, ids=str)
@pytest.mark.parametrize("T,d,f,E,k,cf", [(1, 256, 96, 8, 2, 4.0), (37, 528, 144, 16, 3, 16 / 3), (600, 256, 160, 8, 2, 1.0)])
def test_the_layer_is_its_parts(T, d, f, E, k, cf, rule, dtype):
    say("block", T, d, f, E, k, cf, rule, dtype)
    b = block(T, d, f, E, dtype)
    for residual in (True, False):
        r = call(b, k, cf, residual=residual, eps=1e-5, **rule)
        n = moe.rmsnorm(b["x"], b["norm_weight"], eps=1e-5, residual=b["residual"] if residual else None, mx8=True)
        g = moe.gate(r["logits"], k, bias=b["bias"], **rule)
        e = moe.experts_mx8(n["y8"], g["topk_idx"], g["topk_w"], *b["W"], residual=n["h"], cf=cf)
        same(r, {**n, **g, **e, "logits": r["logits"]})
        y = n["y"].double()
        logits = y @ b["W_router"].double().T
        # sums of d products in fp32, of Gaussian terms: some 2^-24 sqrt(d) of their magnitudes each, which a wrong row passes by far
        size = y.abs() @ b["W_router"].double().abs().T
        assert ((r["logits"] - logits).abs() <= 2.0 ** -24 * (2 * d ** 0.5 + 8) * size).all()
        # the layer in full precision: 8-bit operands are rounded by up to 2^-4, in the mean by 2^-4 / sqrt(12) three times over
        W = [moe.dequantize_mx8(w, torch.float32).double() for w in b["W"]]
        want = n["h"].double()
        for j in range(k):
            e_j = r["topk_idx"][:, j].long()
            keep = (r["slot"][:, j] >= 0).double()[:, None]
            for ex in range(E):
                t = (e_j == ex).nonzero()[:, 0]
                if len(t):
                    gg, uu = y[t] @ W[0][ex].T, y[t] @ W[1][ex].T
                    want[t] += (r["topk_w"][t, j].double()[:, None] * keep[t]) * ((gg * torch.sigmoid(gg) * uu) @ W[2][ex].T)
        part = (want - n["h"].double()).norm()
        assert (r["out"].double() - want).norm() <= 0.08 * part + 2.0 ** -8 * want.norm()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_a_training_step_through_norm_and_gate(score):
    """Gradients of x, residual, the norm's weight and the router of a loss on the weights, the scores and h, against
    autograd in 64 bits with the same choice."""
    T, d, E, k = 50, 96, 24, 4
    b = block(T, d, 32, E, "f32", seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    dw, dsc = torch.randn(T, k, device="cuda", generator=g), 0.1 * torch.randn(T, E, device="cuda", generator=g)
    dres = torch.randn(T, d, device="cuda", generator=g)
    n = moe.rmsnorm(b["x"], b["norm_weight"], residual=b["residual"])
    logits = n["y"] @ b["W_router"].T
    c = moe.gate(logits, k, score=score, bias=b["bias"], groups=4, top_groups=2, group_best=2, scale=1.5)
    dl = moe.gate_backward(logits, c["topk_idx"], dw, score=score, scale=1.5, d_scores=dsc)
    back = moe.rmsnorm_backward(dl @ b["W_router"], n["h"], b["norm_weight"], n["rstd"], dh=dres)
    dWr = dl.T @ n["y"]
    x, res, w, Wr = (b[m].double().requires_grad_() for m in ("x", "residual", "norm_weight", "W_router"))
    h = x + res
    l = (h / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-6) * w) @ Wr.T
    s = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)
    p = s.gather(1, c["topk_idx"].long())
    p = 1.5 * p / p.sum(1, keepdim=True)
    assert (p - c["topk_w"]).abs().max() < 1e-5
    grads = torch.autograd.grad((p * dw).sum() + (s * dsc).sum() + (h * dres).sum(), (x, res, w, Wr))
    for got, want in zip((back["dh"], back["dh"], back["dweight"], dWr), grads):
        assert (got - want).norm() <= 1e-5 * want.norm()   # a few hundred roundings of 2^-24 in a row, of which most cancel


def everything(b, s, stream=None):
    """Every entry point once; s: what earlier calls returned (written again), or empty."""
    kw = dict(stream=stream)
    s["n"] = moe.rmsnorm(b["x"], b["norm_weight"], residual=b["residual"], mx8=True, out=s.get("n"), **kw)
    s["nb"] = moe.rmsnorm_backward(b["residual"], b["x"], b["norm_weight"], b["rstd"], dh=b["x2"], out=s.get("nb"), **kw)
    s["g"] = moe.gate(b["logits"], 4, score="sigmoid", bias=b["bias"], groups=4, top_groups=2, group_best=2, out=s.get("g"), **kw)
    s["gb"] = moe.gate_backward(b["logits"], b["idx"], b["dw"], d_scores=b["dsc"], renormalize=False, out=s.get("gb"), **kw)
    s["e"] = moe.experts_mx8(b["x8"], b["idx"], b["dw"], *b["W"], residual=b["residual"], cf=2.0, out=s.get("e"), **kw)
    s["f"] = moe.forward_mx8(b["x"], b["norm_weight"], b["W_router"], *b["W"], 4, 2.0, residual=b["residual"], out=s.get("f"), **kw)
    return s


def results(s):
    out = {}
    for n, r in s.items():
        for m, t in (r.items() if isinstance(r, dict) else [("", r)]):
            if isinstance(t, moe.Mx8):
                out[n, m] = moe.dequantize_mx8(t, torch.float32)
            elif t is not None and "workspace" not in m and m != "top":
                out[n, m] = t.clone()
    return out


def inputs(T, seed=0):
    b = block(T, 256, 96, 16, seed=seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 100)
    b["x2"] = torch.randn(T, 256, device="cuda", generator=g).bfloat16()
    b["rstd"] = torch.rand(T, device="cuda", generator=g) + 0.5
    b["logits"] = torch.randn(T, 16, device="cuda", generator=g)
    b["idx"] = torch.rand(T, 16, device="cuda", generator=g).topk(4, 1).indices.int()
    b["dw"], b["dsc"] = torch.randn(T, 4, device="cuda", generator=g), torch.randn(T, 16, device="cuda", generator=g)
    b["x8"] = moe.quantize_mx8(b["x2"])
    return b


def refill(b, seed):
    """Other values in the same tensors."""
    o = inputs(b["x"].shape[0], seed)
    for n, t in b.items():
        if n == "W":
            continue
        if isinstance(t, moe.Mx8):
            t.codes.view(torch.uint8).copy_(o[n].codes.view(torch.uint8))
            t.scale.copy_(o[n].scale)
        else:
            t.copy_(o[n])


@pytest.mark.parametrize("T", [1, 40, 700])
def test_another_stream(T):
    b = inputs(T)
    want = results(everything(b, {}))
    other = torch.cuda.Stream()
    busy = torch.randn(2048, 2048, device="cuda")
    for given in (other, other.cuda_stream):
        s = {}
        for again in range(2):   # new tensors, then lent ones
            for _ in range(5):
                busy = busy @ busy / 50   # the current stream is behind
            other.wait_stream(torch.cuda.current_stream())
            everything(b, s, stream=given)
            torch.cuda.current_stream().wait_stream(other)
            got = results(s)
            assert got.keys() == want.keys() and all(torch.equal(got[n], want[n]) for n in want)


@pytest.mark.parametrize("T", [1, 40, 700, 2500])
def test_captured_and_replayed(T):
    """Two graphs with workspaces of their own, replayed in turn on other inputs, with eager work between."""
    bs = [inputs(T, seed) for seed in (0, 1)]
    states, graphs = [{}, {}], []
    for b, s in zip(bs, states):
        everything(b, s)   # the tensors
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            everything(b, s)
        graphs.append(g)
    for turn in range(3):
        for i, (b, s, g) in enumerate(zip(bs, states, graphs)):
            refill(b, 10 * turn + i)
            want = results(everything(b, {}))
            g.replay()
            torch.cuda.synchronize()
            got = results(s)
            assert got.keys() == want.keys()
            for n in want:
                assert torch.equal(got[n], want[n]), (turn, i, n)


def test_lent_results_allocate_nothing():
    b = inputs(40)
    s = everything(b, {})
    torch.cuda.synchronize()
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    everything(b, s)
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before


def test_results_of_other_calls_are_refused():
    b = inputs(8)
    s = everything(b, {})
    for n, f in (("n", lambda o: moe.rmsnorm(b["x"], b["norm_weight"], mx8=True, out=o)),
                 ("nb", lambda o: moe.rmsnorm_backward(b["x"][:4], b["x"][:4], b["norm_weight"], b["rstd"][:4], out=o)),
                 ("f", lambda o: call(b, 4, 1.0, out=o)), ("f", lambda o: call(b, 4, 2.0, residual=False, out=o)),
                 ("e", lambda o: call(b, 4, 2.0, out=o))):
        with pytest.raises(ValueError):
            f(s[n])
        with pytest.raises(ValueError):
            f(dict(s[n]))


@pytest.mark.parametrize("bad", [dict(x=0), dict(norm_weight=0), dict(W_router=0), dict(residual=0), dict(bias=0)], ids=str)
def test_wrong_tensors_are_refused(bad):
    b = block(4, 64, 32, 4)
    name = next(iter(bad))
    t = b[name]
    for wrong in (t.double(), t.cpu(), t[..., :-1], torch.cat([t, t], -1)[..., ::2]):
        with pytest.raises(ValueError):
            call({**b, name: wrong}, 2, 2.0)


def test_no_tokens():
    b = block(0, 64, 32, 4)
    r = call(b, 2, 2.0)
    assert r["out"].shape == (0, 64) and not r["kept_count"].any() and not r["routed_count"].any()
