"""Calls of the few-token layer and the 4-bit weights that a serving loop makes at its edges."""
import pytest

import routing_dispatch_expert_amd as moe
from tests.gpu_util import gpu_available, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(autouse=True)
def _gpu():
    assert gpu_available(), "GPU tests need an MI355X; run them with -m gpu on a GPU host"
    moe.lib()


def weights(dtype, E=8, d=256, f=136):
    g = torch.Generator(device="cuda").manual_seed(4)
    return [(torch.randn(*s, generator=g, device="cuda") * 0.06).to(dtype) for s in ((E, d), (E, f, d), (E, f, d), (E, d, f))]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_empty_batches(dtype):
    """A step without rows returns empty results and zero counts, with a new result and a lent one, on either stream."""
    say(f"empty batches {dtype}")
    wr, *ws = weights(dtype)
    qs = [moe.quantize_q4(w, group=32) for w in ws]
    x = torch.empty(0, 256, dtype=dtype, device="cuda")
    torch.cuda.synchronize()
    for stream in (None, torch.cuda.Stream()):
        for w in (ws, qs):
            r = None
            for _ in range(2):
                r = moe.forward_few(x, wr, *w, k=2, cf=4.0, P=4, out=r, stream=stream)
                torch.cuda.synchronize()
                assert r["C"] == 0 and r["out"].shape == (0, 256) and r["topk_idx"].shape == r["slot"].shape == (0, 2)
                for name, n in (("routed_count", 8), ("kept_count", 8), ("send_count", 4), ("totals", 4)):
                    assert r[name].tolist() == [0] * n, name
        for expert in (None, torch.empty(0, dtype=torch.int32, device="cuda")):
            m = moe.matvec_q4(x, qs[0], expert, stream=stream)
            assert m["out"].shape == (0, 136)
            moe.matvec_q4(x, qs[0], expert, out=m["out"], workspace=m["workspace"], stream=stream)
    torch.cuda.synchronize()


def test_lent_buffers_allocate_nothing():
    """With its results and workspace lent, a call takes no memory: neither from torch nor from the device."""
    for dtype in (torch.bfloat16, torch.float32):
        wr, *ws = weights(dtype)
        qs = [moe.quantize_q4(w, group=64) for w in ws]
        x = torch.randn(5, 256, device="cuda").to(dtype)
        expert = torch.tensor([0, 7, 3, 0, -1], dtype=torch.int32, device="cuda")
        a, b = (moe.forward_few(x, wr, *w, k=2, cf=4.0) for w in (ws, qs))
        m = moe.matvec_q4(x, qs[0], expert)
        torch.cuda.synchronize()
        made, free = torch.cuda.memory_stats()["allocation.all.allocated"], torch.cuda.mem_get_info()[0]
        for _ in range(3):
            moe.forward_few(x, wr, *ws, k=2, cf=4.0, out=a)
            moe.forward_few(x, wr, *qs, k=2, cf=4.0, out=b)
            moe.matvec_q4(x, qs[0], expert, out=m["out"], workspace=m["workspace"])
        torch.cuda.synchronize()
        assert torch.cuda.memory_stats()["allocation.all.allocated"] == made
        assert torch.cuda.mem_get_info()[0] == free


LAYERS = [  # strips of out shared by work-groups and not, two token tiles at a time, many experts, a rank limit
    dict(T=64, d=1032, f=200, E=64, k=8, cf=1.0, dtype="bf16"),
    dict(T=64, d=4360, f=136, E=8, k=4, cf=4.0, dtype="bf16"),
    dict(T=23, d=2056, f=264, E=300, k=6, cf=50.0, dtype="f32"),
    dict(T=64, d=4360, f=136, E=8, k=4, cf=2.0, dtype="bf16", q4=dict(kind="e2m1", group=32)),
    dict(T=17, d=1032, f=520, E=16, k=4, cf=4.0, dtype="f32", q4=dict(kind="u4", group=64), P=8, max_ranks=4),
    dict(T=1, d=7168, f=72, E=256, k=8, cf=32.0, dtype="bf16", q4=dict(kind="u4", group=128)),
]


@pytest.mark.parametrize("case", LAYERS, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items() if k != "q4") +
                         ("-" + c["q4"]["kind"] if "q4" in c else ""))
def test_captured_layers_on_one_workspace(case):
    """Two captured calls with other tokens over one workspace, replayed in turn between eager calls over it."""
    say(f"captured layers {case}")
    c = dict(dict(P=1, max_ranks=0), **case)
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(11)

    def rand(*s, std):
        return (torch.randn(*s, generator=g, device="cuda") * std).to(dt)
    T, d, f, E, k = (c[n] for n in "T d f E k".split())
    wr, ws = rand(E, d, std=d ** -0.5), [rand(E, f, d, std=d ** -0.5), rand(E, f, d, std=d ** -0.5), rand(E, d, f, std=f ** -0.5)]
    if "q4" in c:
        ws = [moe.quantize_q4(w, **c["q4"]) for w in ws]
    bias = rand(E, std=1.0).float()
    n = moe.moe_few_workspace_size(T, d, f, E, k, c["cf"], c["P"], c["dtype"], int("q4" in c))
    ws_mem = torch.empty(n, dtype=torch.uint8, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")

    def made(x):
        st = dict(topk_idx=torch.empty(T, k, **i32), topk_w=torch.empty(T, k, device="cuda"), slot=torch.empty(T, k, **i32),
                  routed_count=torch.empty(E, **i32), kept_count=torch.empty(E, **i32), send_count=torch.empty(c["P"], **i32),
                  totals=torch.empty(4, dtype=torch.int64, device="cuda"))
        out = torch.empty_like(x)
        fn = moe.moe_layer_forward_few_q4 if "q4" in c else moe.moe_layer_forward_few

        def call():
            fn(x, wr, bias, *ws, T, d, f, E, k, c["cf"], c["P"], c["max_ranks"], c["dtype"], out, st, ws_mem, n,
               torch.cuda.current_stream())
        return call, dict(st, out=out)
    calls = [made(rand(T, d, std=1.0)) for _ in range(3)]
    want = []
    for call, o in calls:
        call()
        torch.cuda.synchronize()
        want.append({name: v.clone() for name, v in o.items()})
    graphs = []
    for call, _ in calls[:2]:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call()
    for _ in range(3):
        for i in (0, 1, 1, 0):
            for v in calls[i][1].values():
                v.view(torch.uint8).fill_(0x7f)
            calls[2][0]()
            graphs[i].replay()
            torch.cuda.synchronize()
            for name, v in calls[i][1].items():
                assert torch.equal(v.view(torch.uint8), want[i][name].view(torch.uint8)), name


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_captured_row_products_and_quantiser(dtype):
    say(f"captured row products {dtype}")
    E, N, K, R = 5, 1000, 2312, 37
    g = torch.Generator(device="cuda").manual_seed(12)
    W = torch.randn(E, N, K, generator=g, device="cuda").to(dtype)
    q = moe.quantize_q4(W, group=64)
    x = [torch.randn(R, K, generator=g, device="cuda").to(dtype) for _ in range(2)]
    expert = torch.randint(-1, E + 1, (R,), generator=g, device="cuda", dtype=torch.int32)
    ws = moe.matvec_q4(x[0], q, expert)["workspace"]
    out = [torch.empty(R, N, dtype=dtype, device="cuda") for _ in range(2)]
    codes, scale, zero, back = torch.empty_like(q.codes), torch.empty_like(q.scale), torch.empty_like(q.zero), torch.empty_like(W)
    parts = (codes, scale, zero, "u4", 64)

    def product(i):
        out[i].zero_()
        moe.matvec_q4(x[i], q, expert, out=out[i], workspace=ws)

    def quantiser(_):
        s = torch.cuda.current_stream()
        moe.moe_q4_quantize(W, E, N, K, dtype, parts, s)
        moe.moe_q4_dequantize(parts, E, N, K, dtype, back, s)
    jobs = [(product, 0, (out[0],)), (product, 1, (out[1],)), (quantiser, 0, (codes, scale, zero, back))]
    want, graphs = [], []
    for fn, i, res in jobs:
        fn(i)
        torch.cuda.synchronize()
        want.append([v.clone() for v in res])
    for fn, i, res in jobs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            fn(i)
    for _ in range(3):
        for j, (fn, i, res) in enumerate(jobs):
            for v in res:
                v.view(torch.uint8).fill_(0x7f)
            product(1 - i)
            for v in res:
                v.view(torch.uint8).fill_(0x7f)
            graphs[j].replay()
            torch.cuda.synchronize()
            for v, w in zip(res, want[j]):
                assert torch.equal(v.view(torch.uint8), w.view(torch.uint8))


def test_streams_at_once_on_larger_layers():
    """Calls of three kinds in flight on three streams, a workspace each: every result equals the call's alone."""
    g = torch.Generator(device="cuda").manual_seed(13)

    def rand(*s, std=0.05):
        return (torch.randn(*s, generator=g, device="cuda") * std).bfloat16()
    wr, ws = rand(32, 2048), [rand(32, 512, 2048), rand(32, 512, 2048), rand(32, 2048, 512)]
    qs = [moe.quantize_q4(w, group=32, kind="e2m1") for w in ws]
    xs = [rand(t, 2048, std=1.0) for t in (64, 5, 20)]
    expert = torch.randint(0, 32, (20,), generator=g, device="cuda", dtype=torch.int32)
    kinds = [lambda s, o: moe.forward_few(xs[0], wr, *ws, k=4, cf=8.0, stream=s, out=o),
             lambda s, o: moe.forward_few(xs[1], wr, *qs, k=4, cf=8.0, stream=s, out=o),
             lambda s, o: moe.matvec_q4(xs[2], qs[0], expert, stream=s, **({} if o is None else o))]
    want = [fn(None, None)["out"].clone() for fn in kinds]
    streams = [torch.cuda.Stream() for _ in kinds]
    torch.cuda.synchronize()
    res, got = [None] * 3, [[], [], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            res[i] = kinds[i](s, res[i])
            with torch.cuda.stream(s):
                got[i].append(res[i]["out"].clone())
    torch.cuda.synchronize()
    for i in range(3):
        for o in got[i]:
            assert torch.equal(o.view(torch.int16), want[i].view(torch.int16)), i


def test_lent_result_shows_what_the_call_wrote():
    """Entries of a result that were replaced or taken out hold the later call's outputs, not what was put there."""
    wr, *ws = weights(torch.bfloat16)
    x = [torch.randn(5, 256, device="cuda").bfloat16() for _ in range(2)]
    want = {k: v.clone() for k, v in moe.forward_few(x[1], wr, *ws, k=2, cf=0.5).items() if isinstance(v, torch.Tensor)}
    r = moe.forward_few(x[0], wr, *ws, k=2, cf=0.5)
    r["out"] = r["out"].clone()
    r["topk_w"] = r["topk_w"].double()
    del r["slot"], r["C"]
    r["workspace"] = None
    r["mine"] = 1
    s = moe.forward_few(x[1], wr, *ws, k=2, cf=0.5, out=r)
    torch.cuda.synchronize()
    assert s is r and s["C"] == 1 and s["mine"] == 1
    for name in ("out", "topk_idx", "topk_w", "slot", "routed_count", "kept_count", "send_count", "totals"):
        assert torch.equal(s[name], want[name]), name
