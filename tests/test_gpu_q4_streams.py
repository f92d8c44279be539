"""Calls of the few-token layer and the 4-bit weights on a given stream, next to unfinished work on torch's current one."""
import pytest

import routing_dispatch_expert_amd as moe
from tests.gpu_util import gpu_available, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(autouse=True)
def _gpu():
    assert gpu_available(), "GPU tests need an MI355X; run them with -m gpu on a GPU host"
    moe.lib()


def calls():
    """name -> call(stream), returning a dict of tensors."""
    g = torch.Generator(device="cuda").manual_seed(3)

    def rand(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)
    T, d, f, E, k = 6, 256, 136, 8, 2
    x, wr = rand(T, d), rand(E, d, std=d ** -0.5)
    ws = [rand(E, f, d, std=0.1), rand(E, f, d, std=0.1), rand(E, d, f, std=0.1)]
    qs = [moe.quantize_q4(w, group=64) for w in ws]
    x32, expert = x.float(), torch.tensor([0, 3, -1, 3, 7, 9], dtype=torch.int32, device="cuda")

    def parts(q):
        return {"codes": q.codes, "scale": q.scale, "zero": q.zero}
    return {
        "layer": lambda s: moe.forward_few(x, wr, *ws, k=k, cf=E / k, stream=s),
        "layer_q4": lambda s: moe.forward_few(x, wr, *qs, k=k, cf=E / k, stream=s),
        "matvec": lambda s: moe.matvec_q4(x, qs[0], expert, stream=s),
        "matvec_f32": lambda s: moe.matvec_q4(x32, qs[0], expert, stream=s),
        "quantize": lambda s: parts(moe.quantize_q4(ws[0], group=64, stream=s)),
        "dequantize": lambda s: {"W": moe.dequantize_q4(qs[0], torch.bfloat16, stream=s)},
    }


def tensors(r):
    return {k: v for k, v in r.items() if isinstance(v, torch.Tensor) and k != "workspace"}


@pytest.mark.parametrize("name", ["layer", "layer_q4", "matvec", "matvec_f32", "quantize", "dequantize"])
@pytest.mark.parametrize("raw", [False, True], ids=["stream", "address"])
def test_new_memory_is_not_in_use_elsewhere(name, raw):
    """Work that still waits on the current stream writes and reads memory which torch has taken back: the results of
    a call on another stream must not lie there."""
    say(f"given stream {name} raw={raw}")
    call = calls()[name]
    want = {k: v.clone() for k, v in tensors(call(None)).items()}
    like = {k: v for k, v in call(None).items() if isinstance(v, torch.Tensor)}
    sizes = [v.nbytes for v in like.values()]
    del like
    s = torch.cuda.Stream()
    big = torch.randn(8192, 8192, device="cuda", dtype=torch.bfloat16)
    kept = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda.synchronize()
    temps = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
    for _ in range(30):   # about a millisecond each
        big @ big
    for t, c in zip(temps, kept):
        t.fill_(0x7f)
        c.copy_(t)
    del t, temps
    got = call(s.cuda_stream if raw else s)
    s.synchronize()
    torch.cuda.synchronize()
    got = tensors(got)
    assert got.keys() == want.keys()
    for k in want:
        assert torch.equal(got[k].view(torch.uint8), want[k].view(torch.uint8)), k
    for c in kept:
        assert (c == 0x7f).all()


def test_results_freed_at_once_stay_until_read():
    """A result made on a given stream, read on the current one and dropped: its memory is not handed to the given
    stream's next call while the reading waits."""
    call = calls()["dequantize"]
    want = call(None)["W"].clone()
    s = torch.cuda.Stream()
    big = torch.randn(8192, 8192, device="cuda", dtype=torch.bfloat16)
    torch.cuda.synchronize()
    r = call(s)["W"]
    n = r.numel()
    torch.cuda.current_stream().wait_stream(s)
    for _ in range(30):
        big @ big
    got = r.clone()
    del r
    with torch.cuda.stream(s):
        again = torch.empty(n, dtype=torch.bfloat16, device="cuda").fill_(7)
    torch.cuda.synchronize()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16)) and (again == 7).all()
