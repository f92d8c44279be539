"""The gradients of the layer with a given routing in both types against 64 bits, element by element, with weights of
every size: the weights' gradients do not depend on the weights."""
import numpy as np
import pytest

import routing_dispatch_expert_amd as moe
from tests import routed_reference as ref
from tests.gpu_util import gpu_available, say

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}   # half a step, relative
EDGE = np.float32(2.0 ** -40)
# zeros, subnormal numbers, both sides of the sizes from which a weight is taken late, huge ones
UNUSUAL = [0.0, -0.0, 1e-45, -1e-38, 2.0 ** -126, 1e-30, float(np.nextafter(EDGE, np.float32(0))), float(EDGE), -float(EDGE), 1e-9, 3e5,
           2.0 ** 40, -float(np.nextafter(np.float32(2.0 ** 40), np.float32(np.inf))), 1e20]


@pytest.fixture(autouse=True)
def _gpu():
    assert gpu_available(), "GPU tests need an MI355X; run them with -m gpu on a GPU host"
    moe.lib()


def case(T, d, f, E, k, dtype, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + T)
    rand = lambda *s, std=1.0: (torch.randn(*s, device="cuda", generator=g) * std).to(DT[dtype])  # noqa: E731
    b = dict(x=rand(T, d), W=[rand(E, f, d, std=d ** -0.5), rand(E, f, d, std=d ** -0.5), rand(E, d, f, std=f ** -0.5)], dout=rand(T, d),
             idx=torch.rand(T, E, device="cuda", generator=g).topk(k, 1).indices.int(), w=torch.randn(T, k, device="cuda", generator=g))
    if T > 8 and k > 1:
        b["idx"][1] = b["idx"][1, 0]                             # an expert that a token names twice counts twice
        b["idx"][2, 0], b["idx"][3, 0], b["idx"][4] = -1, E, 1 << 30   # no expert
    return b


def check(b, cf, dtype):
    f = moe.forward_routed(b["x"], b["idx"], b["w"], *b["W"], cf=cf, keep_activations=True)
    got = moe.backward_routed(b["x"], b["idx"], b["w"], *b["W"], b["dout"], cf=cf)
    saved = moe.backward_routed(b["x"], b["idx"], b["w"], *b["W"], b["dout"], cf=cf, saved=f)
    want = ref.gradients(b["x"].double(), b["idx"], b["w"].double(), f["slot"], [m.double() for m in b["W"]], b["dout"].double(),
                         HALF[dtype])
    for n in ("dx", "d_topk_w", "dW_gate", "dW_up", "dW_down"):
        assert torch.equal(got[n], saved[n]), n
        off, most = (got[n].double() - want[n][0]).abs(), want[n][1]
        assert (off <= most).all(), f"{n}: {int((off > most).sum())} of {off.numel()}, up to {(off / most).max()} times"
    # Of eight roundings in a row (g or u, h or the slope, dy, dh twice, dg or du, dX, dx) none is off by more than half a
    # step of its row, and products with Gaussian matrices keep a row's error in proportion; sums of n products in fp32:
    # 2^-23 sqrt(n), five one after the other.
    d, F = b["x"].shape[1], b["W"][0].shape[1]
    part = 8 * HALF[dtype] + 10 * 2.0 ** -24 * max(d, 2 * F) ** 0.5
    off = (got["dx"].double() - want["dx"][0]).norm(dim=1)
    assert (off <= part * want["parts"] + 1e-35).all(), f"dx: {(off / want['parts']).max()}"
    off = (got["d_topk_w"].double() - want["d_topk_w"][0]).norm()
    assert off <= part * want["terms"].norm(), f"d_topk_w: {off / want['terms'].norm()}"   # a sum may be far smaller than its terms
    assert not got["d_topk_w"][f["slot"] < 0].any()
    return f, got


# one token; drops; rows of more than 256 words (in two blocks); an expert's rows by tiles of 256; many experts
SIZES = [(1, 64, 32, 4, 2, 2.0), (60, 104, 72, 5, 3, 0.7), (300, 128, 96, 8, 2, 1.0), (20, 2120, 64, 4, 2, 0.8), (700, 256, 128, 2, 1, 1.5),
         (900, 128, 64, 130, 3, 2.0)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,f,E,k,cf", SIZES)
def test_gradients(T, d, f, E, k, cf, dtype):
    say("routed gradients", T, d, f, E, k, cf, dtype)
    check(case(T, d, f, E, k, dtype), cf, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,f,E,k,cf", SIZES)
def test_weights_of_unusual_size(T, d, f, E, k, cf, dtype):
    say("unusual weights", T, d, f, E, k, cf, dtype)
    b = case(T, d, f, E, k, dtype, seed=1)
    w = b["w"].view(-1)
    at = torch.arange(0, w.numel(), 3 if T > 1 else 1, device="cuda")
    w[at] = torch.tensor(UNUSUAL, device="cuda")[at % len(UNUSUAL)]
    check(b, cf, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_weights_that_are_all_zero(dtype):
    """As a combine weight that is learned from 0 has them: the experts get nothing, the weights their gradient."""
    b = case(200, 128, 64, 8, 2, dtype)
    b["w"].zero_()
    f, got = check(b, 2.0, dtype)
    for n in ("dx", "dW_gate", "dW_up", "dW_down"):
        assert not got[n].any(), n
    assert (got["d_topk_w"][f["slot"] >= 0] != 0).all()


def test_a_weight_of_zero_against_differences():
    """out is linear in a weight: what 1 in place of 0 adds to it, times dout."""
    b = case(40, 128, 64, 4, 2, "f32")
    b["w"][:, 0] = 0
    got = moe.backward_routed(b["x"], b["idx"], b["w"], *b["W"], b["dout"], cf=2.0)["d_topk_w"].double()
    one = b["w"].clone()
    one[:, 0] = 1
    lo, hi = (moe.forward_routed(b["x"], b["idx"], w, *b["W"], cf=2.0)["out"].double() for w in (b["w"], one))
    want = ((hi - lo) * b["dout"].double()).sum(1)
    # out, some units in size, is rounded by 2^-24 of itself twice, in each of 128 terms; sums of 128 in fp32
    assert ((got[:, 0] - want).abs() <= 128 ** 0.5 * 2.0 ** -24 * 64).all()
    assert (got[5:, 0] != 0).all()
