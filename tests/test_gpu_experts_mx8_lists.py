"""The 8-bit experts' lists where the layer's own launches make them (above 8192 copies): indices outside, experts that a
token names twice, drops."""
import numpy as np
import pytest

import routing_dispatch_expert_amd as moe
from tests.gpu_util import gpu_available
from tests.test_gpu_experts_mx8 import route, run_case

pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    assert gpu_available(), "GPU tests need an MI355X; run them with -m gpu on a GPU host"
    moe.lib()


@pytest.mark.parametrize("T,E,k,cf", [(2740, 5, 3, 5 / 3), (2740, 5, 3, 0.6), (4097, 300, 2, 2.0), (1025, 40, 8, 1.0), (8193, 2, 1, 2.0)])
def test_outside_and_repeated_indices(T, E, k, cf):
    assert T * k > 8192
    rng = np.random.default_rng(T + E)
    idx = route(rng, T, E, k)
    idx[0] = np.resize((-1, E, 1 << 30), k)      # no expert at all
    idx[1] = E - 1
    idx[2::3, k - 1] = -(1 << 31)
    idx[T - 1] = idx[T - 1, 0]
    run_case(T, 16, 16, E, k, cf, idx=idx)
