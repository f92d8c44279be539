"""What an expert returns is summed over a token's experts in fp32 and rounded once, with the residual: y's own rounding
to bf16 would be as large as the output's."""
import numpy as np
import pytest

import routing_dispatch_expert_amd as moe
from tests import mx8_reference as ref
from tests.gpu_util import gpu_available, say

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    assert gpu_available(), "GPU tests need an MI355X; run them with -m gpu on a GPU host"
    moe.lib()


# strips, tiles of 128 rows and of 256, down's tiles split over K
@pytest.mark.parametrize("T,f", [(3, 160), (40, 160), (300, 160), (300, 6144), (60, 6144)])
def test_one_rounding(T, f):
    """Two experts whose y cancel but for some 2^-8 of them. y is a sum of whole numbers below 2^24 (exact, but for what an
    instruction cuts off: 2^-12 at most); in bf16 each would be off by up to 2^-8."""
    say("one rounding", T, f)
    d = 256
    rng = np.random.default_rng(T + f)
    # g = 32 and 33 (silu(g) = g in fp32), u = 1: h = 32 for all features, in 8 bits as it is
    x = np.zeros((T, d))
    x[:, 0], x[:, 1] = 32, 1
    Wg, Wu = np.zeros((2, f, d)), np.zeros((2, f, d))
    Wg[:, :, 0], Wu[:, :, 1] = 1, 1
    Wd = np.zeros((2, d, f))
    Wd[0] = rng.integers(0, 16, (d, f))
    Wd[1] = -Wd[0]
    Wd[1] += rng.integers(-1, 2, (d, f))     # codes up to 16 are whole numbers

    def mx(a):
        q = torch.from_numpy(a).to(torch.float8_e4m3fn).cuda()
        assert np.array_equal(q.double().cpu().numpy(), a)
        return moe.Mx8(q, torch.full((*a.shape[:-2], -(-a.shape[-1] // 128), a.shape[-2], 4), 127, dtype=torch.uint8, device="cuda"))

    idx = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda").expand(T, 2).contiguous()
    w = torch.ones(T, 2, device="cuda")
    residual = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    y = 32 * Wd.sum(2)
    off = 2.0 ** -12 * np.abs(y).sum(0)
    assert np.abs(y).max() < 2.0 ** 24 and (off < 2.0 ** -10 * np.abs(y).min()).all()
    r = moe.experts_mx8(mx(x), idx, w, mx(Wg), mx(Wu), mx(Wd), residual, 1.0)["out"].double().cpu().numpy()
    want = y.sum(0)
    bad = np.abs(r - want) > off + 2.0 ** -8 * (np.abs(want) + off)
    assert not bad.any(), f"{bad.sum()} of {bad.size}, up to {(np.abs(r - want) / off).max()} times"
    # what y in bf16 would give is told apart
    rounded = torch.from_numpy(y).to(torch.bfloat16).double().numpy().sum(0)
    assert (np.abs(rounded - want) > off + 2.0 ** -8 * (np.abs(want) + off)).mean() > 0.2
