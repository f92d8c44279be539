"""The few-token layer's choice of experts where their scores nearly agree."""
import numpy as np
import pytest

import routing_dispatch_expert_amd as moe
from tests.gpu_util import gpu_available, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(autouse=True)
def _gpu():
    assert gpu_available(), "GPU tests need an MI355X; run them with -m gpu on a GPU host"
    moe.lib()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,d,E,k", [(1, 8, 8, 2), (1, 7168, 256, 8), (4, 520, 16, 4), (33, 1032, 60, 6), (64, 2048, 256, 8)])
def test_scores_far_closer_than_fp32_rounds(T, d, E, k, dtype):
    """All experts' rows are alike but for one column, which moves their scores apart by 2^-30 where the scores are
    about 1 (fp32 rounds there to 2^-24). In fp64 a sum of d products is off by at most (d + 16) 2^-53 of their
    magnitudes' sum, below 2^-33 here, so the order is the column's."""
    say(f"close scores T={T} d={d} E={E} {dtype}")
    g = torch.Generator().manual_seed(T + d)
    x = torch.randn(T, d, generator=g).to(dtype)
    row = (torch.randn(d, generator=g) / d ** 0.5).to(dtype)
    order = torch.randperm(E, generator=g)   # whole numbers up to 255: exact in bf16
    at = d // 2
    x[:, at] = 2.0 ** -30
    x[1::2, at] *= -1
    W = row.repeat(E, 1)
    W[:, at] = order.to(dtype)
    mag = (x.double().abs() @ W.double().abs().T).max().item()
    assert (d + 16) * 2.0 ** -53 * mag < 2.0 ** -33
    f = 16
    ws = [torch.zeros(s, dtype=dtype, device="cuda") for s in ((E, f, d), (E, f, d), (E, d, f))]
    r = moe.forward_few(x.cuda(), W.cuda(), *ws, k=k, cf=E / k)
    up = np.argsort(-order.numpy())[:k]
    down = np.argsort(order.numpy())[:k]
    want = np.stack([down if t % 2 else up for t in range(T)])
    assert np.array_equal(r["topk_idx"].cpu().numpy(), want)
    assert (r["topk_w"].cpu() - 1 / k).abs().max() <= 2.0 ** -22
