"""The norm's weight gradient against 64 bits, with a bound from the number of additions that its sums have."""
import numpy as np
import pytest

import routing_dispatch_expert_amd as moe
from tests.gpu_util import U, gpu_available, say
from tests.test_gpu_mx8 import BACK, HALF, dev, host, rows

pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    assert gpu_available(), "GPU tests need an MI355X; run them with -m gpu on a GPU host"
    moe.lib()


def additions(R, d, dtype):
    """Most additions in a row: a share's rows, its four waves (narrow rows), a slice's shares, the 32 slices."""
    words = d // (8 if dtype == "bf16" else 4)
    if words <= 256:
        shares, takers = min(-(-R // 4), 512), 4
    else:
        shares, takers = min(R, 512 if words <= 2048 else 256), 1
    return -(-R // (shares * takers)) + takers - 1 + -(-shares // 32) + 32


@pytest.mark.parametrize("dtype,R,d", [(t, *s) for t in BACK for s in BACK[t]] + [("bf16", 5000, 512), ("f32", 3000, 2080)])
def test_dweight(dtype, R, d):
    say("norm's dweight", dtype, R, d)
    rng = np.random.default_rng(R + d + 1)
    h, w, dy = rows(rng, R, d, dtype), dev(1 + 0.2 * rng.standard_normal(d), dtype), dev(rng.standard_normal((R, d)), dtype)
    rstd = moe.rmsnorm(h, w)["rstd"]
    got = host(moe.rmsnorm_backward(dy, h, w, rstd)["dweight"])
    terms = host(dy) * host(h) * host(rstd)[:, None]
    off = U * (additions(R, d, dtype) + 2) * np.abs(terms).sum(0)   # and a term's two products
    want = terms.sum(0)
    assert np.all(np.abs(got - want) <= off + HALF[dtype] * (np.abs(want) + off))
