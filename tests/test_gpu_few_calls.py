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
