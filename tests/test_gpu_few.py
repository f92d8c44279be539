"""The layer for few tokens (moe_layer_forward_few and its 4-bit form) on the
GPU, against 64 bits and the bound derived in few_reference.py; its routing
outputs exactly. Every output and the workspace is followed by a canary."""
import numpy as np
import pytest

import moe_inputs
import routing_dispatch_expert_amd as moe
from tests import few_reference as ref
from tests.gpu_util import Guarded, bits_to_f64, gpu_available, say, to_dev, to_host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(autouse=True)
def _gpu():
    assert gpu_available(), "GPU tests need an MI355X; run them with -m gpu on a GPU host"
    moe.lib()


class Q4:
    """4-bit weights of one matrix stack: on the device, and decoded per expert in 64 bits."""

    def __init__(self, rng, E, N, K, group, kind, zero_points):
        codes, scale, zero = ref.random_q4(rng, E, N, K, group, kind, zero_points)
        z = None if zero is None else torch.from_numpy(zero).cuda()
        self.dev = moe.Q4Weights(torch.from_numpy(codes).cuda(), to_dev(scale, "bf16"), z, (E, N, K), group, kind)
        s64 = moe_inputs.bits_to_f64(scale, "bf16")
        self.expert = lambda e: tuple(v[0] for v in ref.q4_decode(
            codes[e:e + 1], s64[e:e + 1], None if zero is None else zero[e:e + 1], (1, N, K), group, kind))


def weights_of(wl, q4=None):
    """(device gate, up, down) and the 64-bit view that few_reference.layer takes."""
    if q4:
        rng = np.random.default_rng(wl.seed + 1)
        E, d, f = wl.E, wl.d, wl.d_ff
        ws = [Q4(rng, E, f, d, **q4), Q4(rng, E, f, d, **q4), Q4(rng, E, d, f, **q4)]
        return [w.dev for w in ws], dict(zip("gud", (w.expert for w in ws)))
    host = wl.all_expert_weights()

    def view(a):
        def one(e):
            v = bits_to_f64(a[e], wl.dtype)
            return v, np.abs(v)
        return one
    return [to_dev(a, wl.dtype) for a in host], dict(zip("gud", (view(a) for a in host)))


def few_outputs(wl, x, g):
    i32 = torch.int32
    return {"out": g.empty((wl.T, wl.d), x.dtype, "out"), "topk_idx": g.empty((wl.T, wl.k), i32, "topk_idx"),
            "topk_w": g.empty((wl.T, wl.k), torch.float32, "topk_w"), "slot": g.empty((wl.T, wl.k), i32, "slot"),
            "routed_count": g.empty((wl.E,), i32, "routed"), "kept_count": g.empty((wl.E,), i32, "kept"),
            "send_count": g.empty((wl.P,), i32, "send"), "totals": g.empty((4,), torch.int64, "totals")}


def call_few(wl, x, wr, b, dev, o, ws, n, stream=None, stats=True):
    fn = moe.moe_layer_forward_few_q4 if isinstance(dev[0], moe.Q4Weights) else moe.moe_layer_forward_few
    st = {k: v for k, v in o.items() if k != "out"} if stats else None
    fn(x, wr, b, *dev, wl.T, wl.d, wl.d_ff, wl.E, wl.k, wl.cf, wl.P, wl.max_ranks, wl.dtype, o["out"], st, ws, n, stream)


def run_few(wl, dev, stats=True):
    x, wr = to_dev(wl.x, wl.dtype), to_dev(wl.wr, wl.dtype)
    b = None if wl.bias_vec is None else torch.from_numpy(wl.bias_vec).cuda()
    g = Guarded()
    o = few_outputs(wl, x, g)
    n = moe.moe_few_workspace_size(wl.T, wl.d, wl.d_ff, wl.E, wl.k, wl.cf, wl.P, wl.dtype,
                                   int(isinstance(dev[0], moe.Q4Weights)))
    ws = g.empty((-(-n // 4),), torch.int32, "workspace")
    ws.fill_(-1)   # whatever the workspace holds
    call_few(wl, x, wr, b, dev, o, ws, n, stats=stats)
    torch.cuda.synchronize()
    g.check()
    return o


def check(wl, o, view):
    r = ref.routing(wl)
    for key, want in (("topk_idx", r["idx"]), ("slot", r["slot"]), ("routed_count", r["routed"]),
                      ("kept_count", r["kept"]), ("send_count", r["send"])):
        assert np.array_equal(o[key].cpu().numpy(), want), key
    assert o["totals"].tolist() == r["totals"]
    w = o["topk_w"].cpu().numpy().astype(np.float64)
    assert (np.abs(w - r["w"]) <= r["w_err"] * r["w"] + 1e-30).all(), "topk_w"
    want, bound = ref.layer(wl, view, r)
    got = bits_to_f64(to_host(o["out"], wl.dtype), wl.dtype)
    off = np.abs(got - want) / bound
    say(f"  out: largest error {off.max():.3f} of its bound")
    assert off.max() <= 1, f"out: {off.max()} of its bound at {np.unravel_index(off.argmax(), off.shape)}"
    return r


def wl_of(**c):
    c.setdefault("seed", 31)
    c.setdefault("wr_std", 1 / np.sqrt(c["d"]))
    return moe_inputs.custom(**c)


U4 = dict(kind="u4", group=128, zero_points=True)
CASES = [
    # one token; the smallest widths; one expert
    dict(T=1, d=8, E=1, k=1, d_ff=8, cf=1.0),
    dict(T=1, d=256, E=16, k=4, d_ff=128, cf=4.0),
    dict(T=1, d=1032, E=256, k=8, d_ff=72, cf=2.0, P=8),
    # odd counts, ragged widths, drops
    dict(T=3, d=136, E=12, k=3, d_ff=88, cf=0.5, P=4),
    dict(T=7, d=520, E=6, k=2, d_ff=264, cf=0.25, P=2),
    # around the 16-token tiles: every token to expert 0 (kept 15, 16, 17, 33, 64)
    dict(T=15, d=64, E=4, k=1, d_ff=48, cf=4.0, bias="hot0"),
    dict(T=16, d=64, E=4, k=1, d_ff=48, cf=4.0, bias="hot0"),
    dict(T=17, d=64, E=4, k=1, d_ff=48, cf=4.0, bias="hot0"),
    dict(T=33, d=64, E=4, k=2, d_ff=48, cf=2.0, bias="hot0"),
    dict(T=64, d=72, E=4, k=4, d_ff=136, cf=1.0, P=2),
    # hot expert over its capacity: fully dropped tokens
    dict(T=64, d=64, E=8, k=1, d_ff=64, cf=0.5, bias="hot0", P=4),
    # rank limit, a bias, many experts, many choices
    dict(T=20, d=128, E=64, k=6, d_ff=64, cf=1.0, P=8, max_ranks=2, bias="zipf1.2"),
    dict(T=5, d=64, E=1024, k=32, d_ff=32, cf=4.0, P=128),
    dict(T=64, d=64, E=320, k=8, d_ff=32, cf=1.0, P=64, max_ranks=5),
    dict(T=64, d=64, E=96, k=20, d_ff=32, cf=1.0, P=3),
]


# what the sizes above do not reach: many feature strips a work-group of 4, 2 and 1 waves each; contractions of several
# staged runs a wave; more than 256 strips of out; both sides of 64 copies and of 64 ranks
LONG = [
    dict(T=64, d=136, E=64, k=8, d_ff=200, cf=2.0),
    dict(T=64, d=264, E=64, k=8, d_ff=392, cf=1.0, P=2),
    dict(T=3, d=72, E=1, k=1, d_ff=262168, cf=1.0),
    dict(T=3, d=4360, E=4, k=2, d_ff=136, cf=2.0),
    dict(T=40, d=4360, E=4, k=2, d_ff=72, cf=2.0),
    dict(T=16, d=136, E=16, k=4, d_ff=136, cf=1.0),
    dict(T=13, d=136, E=16, k=5, d_ff=136, cf=1.0),
    dict(T=2, d=136, E=1024, k=4, d_ff=16, cf=2.0, P=128),
]


def _id(c):
    return "-".join(f"{k}{v}" for k, v in c.items())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=_id)
def test_few_layer(case, dtype):
    say(f"few layer {dtype} {case}")
    wl = wl_of(dtype=dtype, **case)
    dev, view = weights_of(wl)
    check(wl, run_few(wl, dev), view)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q4", [U4, dict(U4, group=64), dict(U4, group=32, zero_points=False),
                                dict(kind="e2m1", group=32, zero_points=False),
                                dict(kind="e2m1", group=64, zero_points=False),
                                dict(kind="e2m1", group=128, zero_points=False)], ids=_id)
@pytest.mark.parametrize("case", [CASES[i] for i in (0, 2, 3, 4, 7, 9, 11)], ids=_id)
def test_few_layer_q4(case, q4, dtype):
    say(f"few layer {dtype} {q4} {case}")
    wl = wl_of(dtype=dtype, **case)
    dev, view = weights_of(wl, q4)
    check(wl, run_few(wl, dev), view)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", LONG, ids=_id)
def test_few_layer_many_strips_and_long_rows(case, dtype):
    say(f"few layer {dtype} {case}")
    wl = wl_of(dtype=dtype, **case)
    dev, view = weights_of(wl)
    check(wl, run_few(wl, dev), view)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q4", [dict(U4, group=64), dict(kind="e2m1", group=32, zero_points=False)], ids=_id)
@pytest.mark.parametrize("case", [LONG[i] for i in (0, 1, 3, 4)] + [
    dict(T=1, d=16520, E=2, k=1, d_ff=40, cf=2.0),
    dict(T=6, d=40, E=2, k=2, d_ff=16520, cf=2.0),
    dict(T=3, d=24, E=1, k=1, d_ff=262168, cf=1.0),
], ids=_id)
def test_few_layer_q4_many_strips_and_long_rows(case, q4, dtype):
    say(f"few layer {dtype} {q4} {case}")
    wl = wl_of(dtype=dtype, **case)
    dev, view = weights_of(wl, q4)
    check(wl, run_few(wl, dev), view)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,f", [(136, 72), (8, 24), (392, 200), (1032, 40)])
def test_weights_not_chosen_may_hold_anything(d, f, dtype):
    """NaN and infinities in the matrices of experts without copies change nothing (rows end inside a cache line that
    the next expert's first row shares), and in one row of W_down only that column of out."""
    wl = wl_of(T=9, d=d, E=3, k=1, d_ff=f, cf=3.0, dtype=dtype)
    x, wr = to_dev(wl.x, dtype), to_dev(wl.wr, dtype)
    bias = torch.tensor([0.0, 1e4, 0.0], device="cuda")
    dev, _ = weights_of(wl)
    want = moe.forward_few(x, wr, *dev, k=1, cf=3.0, router_bias=bias)["out"].clone()
    assert torch.isfinite(want).all()
    for bad in (float("nan"), float("inf")):
        spoilt = [w.clone() for w in dev]
        for w in spoilt:
            w[0] = w[2] = bad
        got = moe.forward_few(x, wr, *spoilt, k=1, cf=3.0, router_bias=bias)["out"]
        assert torch.equal(got, want)
        spoilt[2][1, 5] = bad
        got = moe.forward_few(x, wr, *spoilt, k=1, cf=3.0, router_bias=bias)["out"]
        rest = [c for c in range(d) if c != 5]
        assert torch.equal(got[:, rest], want[:, rest]) and not torch.isfinite(got[:, 5]).any()


def test_without_stats():
    wl = wl_of(T=6, d=256, E=8, k=2, d_ff=128, cf=0.5, dtype="bf16")
    dev, _ = weights_of(wl)
    a, b = run_few(wl, dev), run_few(wl, dev, stats=False)
    assert torch.equal(a["out"].view(torch.int16), b["out"].view(torch.int16))


@pytest.mark.parametrize("dtype,q4", [("bf16", None), ("f32", None), ("bf16", U4), ("f32", dict(U4, group=32))])
def test_agrees_with_the_layer(dtype, q4):
    """Same choices, slots and counts as moe_layer_forward, and outputs within the sum of both errors."""
    wl = wl_of(T=48, d=512, E=32, k=4, d_ff=384, cf=1.0, P=4, dtype=dtype)
    dev, _ = weights_of(wl, q4)
    x, wr = to_dev(wl.x, dtype), to_dev(wl.wr, dtype)
    few = moe.forward_few(x, wr, *dev, k=wl.k, cf=wl.cf, P=wl.P)
    wide = [moe.dequantize_q4(w, x.dtype) for w in dev] if q4 else dev   # bf16: one more rounding of the weights
    full = moe.forward(x, wr, *wide, k=wl.k, cf=wl.cf, P=wl.P)
    for key in ("topk_idx", "slot", "routed_count", "kept_count", "send_count", "totals"):
        assert torch.equal(few[key], full[key]), key
    a, b = few["out"].double(), full["out"].double()
    # bf16: h, y, out and, in 4 bits, the three matrices are rounded on the other path: at most 8 steps of
    # 2^-8 on an expert's share, which stays under the row's largest value
    tol = 8 * 2.0 ** -8 if dtype == "bf16" else 1e-4
    assert ((a - b).abs().amax(1) <= tol * b.abs().amax(1)).all()


@pytest.mark.parametrize("q4", [None, U4, dict(kind="e2m1", group=32, zero_points=False)], ids=str)
def test_nan_token_spoils_no_other(q4):
    """A token of NaN (or infinities) gets distinct experts inside [0, E) and changes no other token's output."""
    wl = wl_of(T=9, d=136, E=8, k=2, d_ff=64, cf=4.0, dtype="bf16")   # C = T: nothing is dropped
    dev, _ = weights_of(wl, q4)
    x, wr = to_dev(wl.x, "bf16"), to_dev(wl.wr, "bf16")
    want = moe.forward_few(x, wr, *dev, k=2, cf=4.0)["out"].clone()
    for bad in (float("nan"), float("inf"), -float("inf")):
        y = x.clone()
        y[4] = bad
        r = moe.forward_few(y, wr, *dev, k=2, cf=4.0)
        torch.cuda.synchronize()
        idx = r["topk_idx"][4].tolist()
        assert len(set(idx)) == 2 and all(0 <= e < 8 for e in idx)
        rest = [t for t in range(9) if t != 4]
        assert torch.equal(r["out"][rest].view(torch.int16), want[rest].view(torch.int16))


def _bits(o):
    return {k: v.contiguous().view(torch.uint8).clone() for k, v in o.items()}


@pytest.mark.parametrize("dtype,q4", [("bf16", None), ("f32", dict(U4, group=64))], ids=str)
def test_two_captured_calls_share_a_workspace(dtype, q4):
    """Two captured calls over one workspace, replayed in turn with eager calls of other sizes between them."""
    say(f"few layer graphs {dtype} {q4}")
    wls = [wl_of(T=9, d=256, E=16, k=4, d_ff=192, cf=1.0, P=2, dtype=dtype, seed=5),
           wl_of(T=64, d=256, E=16, k=2, d_ff=192, cf=0.5, P=2, dtype=dtype, seed=6)]
    dev, view = weights_of(wls[0], q4)
    other = wl_of(T=2, d=256, E=16, k=1, d_ff=192, cf=2.0, P=2, dtype=dtype, seed=7)
    sizes = [moe.moe_few_workspace_size(w.T, w.d, w.d_ff, w.E, w.k, w.cf, w.P, dtype, int(bool(q4)))
             for w in (*wls, other)]
    ws = torch.empty(max(sizes), dtype=torch.uint8, device="cuda")
    made = []
    for wl, n in zip((*wls, other), sizes):
        x, wr = to_dev(wl.x, dtype), to_dev(wl.wr, dtype)
        o = {k: v for k, v in few_outputs(wl, x, Guarded()).items()}
        made.append((wl, x, wr, o, n))

    def call(m, stream=None):
        call_few(m[0], m[1], m[2], None, dev, m[3], ws, m[4], stream)

    want = []
    for m in made[:2]:
        call(m)
        torch.cuda.synchronize()
        want.append(_bits(m[3]))
    graphs = []
    for m in made[:2]:
        g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=s):
            call(m, torch.cuda.current_stream())
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(3):
        for i in (0, 1, 1, 0):
            for v in made[i][3].values():
                v.view(torch.uint8).fill_(0x7f)
            call(made[2])
            torch.cuda.synchronize()
            graphs[i].replay()
            torch.cuda.synchronize()
            for k, v in _bits(made[i][3]).items():
                assert torch.equal(v, want[i][k]), k


def test_two_streams_at_once():
    """Calls in flight on two streams, a workspace each, repeated: every result equals the call's alone."""
    wls = [wl_of(T=t, d=512, E=32, k=4, d_ff=256, cf=2.0, dtype="bf16", seed=s) for t, s in ((33, 8), (1, 9))]
    dev, _ = weights_of(wls[0])
    ins = [(to_dev(w.x, "bf16"), to_dev(w.wr, "bf16")) for w in wls]
    want = [moe.forward_few(x, wr, *dev, k=4, cf=2.0)["out"].clone() for x, wr in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    res = [None, None]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            res[i] = moe.forward_few(*ins[i], *dev, k=4, cf=2.0, stream=s, out=res[i])
            with torch.cuda.stream(s):
                got[i].append(res[i]["out"].clone())
    torch.cuda.synchronize()
    for i in range(2):
        for o in got[i]:
            assert torch.equal(o.view(torch.int16), want[i].view(torch.int16))


def test_current_stream_is_the_default():
    """Without a stream the call runs on torch's current one: it sees what was written there just before."""
    wl = wl_of(T=4, d=256, E=8, k=2, d_ff=128, cf=4.0, dtype="bf16")
    dev, _ = weights_of(wl)
    x, wr = to_dev(wl.x, "bf16"), to_dev(wl.wr, "bf16")
    want = moe.forward_few(x, wr, *dev, k=2, cf=4.0)["out"].clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        y = torch.zeros_like(x)
        y.copy_(x)
        r = moe.forward_few(y, wr, *dev, k=2, cf=4.0)
        got = r["out"].clone()
    torch.cuda.synchronize()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dropped_tokens_pass_bit_for_bit(dtype):
    """Zeros of either sign, infinities and NaN of tokens without a kept copy, as moe_layer_forward passes them."""
    for d, q4 in ((136, None), (4360, None), (136, U4)):   # strips shared by work-groups, and not
        wl = wl_of(T=12, d=d, E=4, k=1, d_ff=64, cf=1.0, dtype=dtype, bias="hot0", reject=False)
        dev, _ = weights_of(wl, q4)
        x, wr = to_dev(wl.x, dtype), to_dev(wl.wr, dtype)
        bits = x.view(torch.int16 if dtype == "bf16" else torch.int32)
        bits[5:, 1::4] = bits.new_tensor(-2 ** (15 if dtype == "bf16" else 31))   # -0.0
        bits[5:, 2::4] = 0
        few = moe.forward_few(x, torch.zeros_like(wr), *dev, k=1, cf=1.0, router_bias=torch.from_numpy(wl.bias_vec).cuda())
        bits[7, 3], bits[8, 3], bits[9, 3] = (0x7f81, -0x80, 0x7f80) if dtype == "bf16" else (0x7f800001, -0x800000, 0x7f800000)
        few = moe.forward_few(x, torch.zeros_like(wr), *dev, k=1, cf=1.0, router_bias=torch.from_numpy(wl.bias_vec).cuda())
        torch.cuda.synchronize()
        lost = (few["slot"] < 0).all(1)
        # NaN scores choose what they like; the others' first C = 3 stay, and every later token is lost
        assert lost[[5, 6, 10, 11]].all()
        assert torch.equal(few["out"].view(bits.dtype)[lost], bits[lost])


def test_lent_buffers_on_another_stream():
    """Buffers lent to a call on a given stream stay its own until it is done, also when dropped at once."""
    wl = wl_of(T=8, d=512, E=16, k=4, d_ff=512, cf=4.0, dtype="bf16")
    dev, _ = weights_of(wl)
    x, wr = to_dev(wl.x, "bf16"), to_dev(wl.wr, "bf16")
    want = moe.forward_few(x, wr, *dev, k=4, cf=4.0)["out"].clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        r = moe.forward_few(x, wr, *dev, k=4, cf=4.0)
        s.wait_stream(torch.cuda.current_stream())
        r = moe.forward_few(x, wr, *dev, k=4, cf=4.0, stream=s, out=r)
        with torch.cuda.stream(s):
            got = r["out"].clone()
        n = r["workspace"].numel()
        y = x.clone()
        s.wait_stream(torch.cuda.current_stream())
        r = moe.forward_few(y, wr, *dev, k=4, cf=4.0, stream=s, router_bias=None)
        with torch.cuda.stream(s):
            again = r["out"].clone()
        del y
        torch.empty_like(x).fill_(7)   # must not get y's memory while the call runs
        del r
        torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0x7f)
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
        assert torch.equal(again.view(torch.int16), want.view(torch.int16))


def test_results_lend_their_buffers():
    wl = wl_of(T=5, d=128, E=8, k=2, d_ff=64, cf=4.0, dtype="bf16")
    dev, _ = weights_of(wl)
    x, wr = to_dev(wl.x, "bf16"), to_dev(wl.wr, "bf16")
    a = moe.forward_few(x, wr, *dev, k=2, cf=4.0)
    first = a["out"].clone()
    b = moe.forward_few(x.flip(0).contiguous(), wr, *dev, k=2, cf=4.0, out=a)
    assert b is a and b["out"].data_ptr() == a["out"].data_ptr()
    torch.cuda.synchronize()
    assert torch.equal(b["out"].flip(0).view(torch.int16), first.view(torch.int16))
    with pytest.raises(ValueError):
        moe.forward_few(x[:4], wr, *dev, k=2, cf=4.0, out=a)
    with pytest.raises(ValueError):
        moe.forward_few(x, wr, *dev, k=2, cf=4.0, out=dict(a))


def test_decoding_with_quantized_weights():
    """As a server uses them together: weights quantised once, a prompt through the wide layer on the dequantised
    weights, then single tokens through the few-token layer, each step's output the next one's input, with an
    output projection in 4 bits after it. Every step is held to the 64-bit layer on the step's own input."""
    say("decode with quantised weights")
    wl = wl_of(T=4, d=256, E=8, k=2, d_ff=384, cf=4.0, dtype="bf16", seed=12)
    host, _ = weights_of(wl)
    q = [moe.quantize_q4(w, group=64, kind="u4") for w in host]
    head = moe.quantize_q4(torch.randn(1, 320, 256, device="cuda", dtype=torch.bfloat16), group=32, kind="e2m1")

    def decoded(w):
        c, s, z = (None if t is None else t for t in (w.codes.cpu().numpy(), to_host(w.scale, "bf16"), w.zero))
        W, A = ref.q4_decode(c, moe_inputs.bits_to_f64(s, "bf16"), None if z is None else z.cpu().numpy(), w.shape,
                             w.group, w.kind)
        return lambda e: (W[e], A[e])
    view, hv = dict(zip("gud", map(decoded, q))), decoded(head)
    prompt = moe.forward(to_dev(wl.x, "bf16"), to_dev(wl.wr, "bf16"), *(moe.dequantize_q4(w, torch.bfloat16) for w in q),
                         k=2, cf=4.0)["out"]
    x, wr, res = prompt[-1:].clone(), to_dev(wl.wr, "bf16"), None
    for step in range(4):
        one = wl_of(T=1, d=256, E=8, k=2, d_ff=384, cf=4.0, dtype="bf16", seed=12)
        one.x = to_host(x, "bf16")
        res = moe.forward_few(x, wr, *q, k=2, cf=4.0, out=res)
        logits = moe.matvec_q4(res["out"], head)["out"]
        torch.cuda.synchronize()
        r = ref.routing(one)
        assert np.array_equal(res["topk_idx"].cpu().numpy(), r["idx"])
        want, bound = ref.layer(one, view, r)
        got = bits_to_f64(to_host(res["out"], "bf16"), "bf16")
        assert (np.abs(got - want) <= bound).all(), step
        W, A = hv(0)
        lw = got @ W.T
        assert (np.abs(bits_to_f64(to_host(logits, "bf16"), "bf16") - lw) <=
                2.0 ** -8 * np.abs(lw) + 1.01 * 264 * ref.ACC * (np.abs(got) @ A.T) + 1e-30).all()
        x = res["out"].clone()
