"""The few-token layer and the row products on either side of the row length from which eight waves share a pair of
strips (40 tiles of 128 columns in 4 bits, 80 lines of 128 bytes else), against 64 bits."""
import numpy as np
import pytest

import moe_inputs
import routing_dispatch_expert_amd as moe
from tests import few_reference as ref
from tests.gpu_util import bits_to_f64, gpu_available, say, to_dev, to_host
from tests.test_gpu_few import U4, check, run_few, weights_of, wl_of

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
E2M1 = dict(kind="e2m1", group=32, zero_points=False)


@pytest.fixture(autouse=True)
def _gpu():
    assert gpu_available(), "GPU tests need an MI355X; run them with -m gpu on a GPU host"
    moe.lib()


@pytest.mark.parametrize("dtype,d", [("bf16", 5056), ("bf16", 5064), ("bf16", 7176), ("f32", 2528), ("f32", 2532),
                                     ("f32", 4100)])
@pytest.mark.parametrize("T,cf", [(1, 4.0), (7, 4.0), (40, 1.0)])
def test_few_layer(T, cf, dtype, d):
    say(f"few layer {dtype} T={T} d={d}")
    wl = wl_of(T=T, d=d, E=4, k=2 if T < 40 else 1, d_ff=40, cf=cf, dtype=dtype)
    dev, view = weights_of(wl)
    check(wl, run_few(wl, dev), view)


@pytest.mark.parametrize("q4", [U4, E2M1], ids=["u4", "e2m1"])
@pytest.mark.parametrize("d", [4992, 5000, 5128])
@pytest.mark.parametrize("T,dtype", [(1, "bf16"), (5, "bf16"), (20, "bf16"), (5, "f32")])
def test_few_layer_q4(T, dtype, d, q4):
    say(f"few layer {dtype} {q4} T={T} d={d}")
    wl = wl_of(T=T, d=d, E=4, k=2, d_ff=40, cf=2.0, dtype=dtype)
    dev, view = weights_of(wl, q4)
    check(wl, run_few(wl, dev), view)


@pytest.mark.parametrize("kind,group", [("u4", 128), ("u4", 32), ("e2m1", 64)])
@pytest.mark.parametrize("K", [4992, 5000, 5128])
@pytest.mark.parametrize("R,E", [(1, 1), (6, 3), (33, 2)])
def test_row_products(R, E, K, kind, group):
    say(f"matvec R={R} E={E} K={K} {kind} {group}")
    N = 72
    rng = np.random.default_rng(R + K)
    codes, scale, z = ref.random_q4(rng, E, N, K, group, kind, True)
    host = moe_inputs.to_bf16_bits(rng.standard_normal((R, K)).astype(np.float32))
    expert = rng.integers(0, E, R).astype(np.int32)
    q = moe.Q4Weights(torch.from_numpy(codes).cuda(), to_dev(scale, "bf16"), None if z is None else torch.from_numpy(z).cuda(),
                      (E, N, K), group, kind)
    out = moe.matvec_q4(to_dev(host, "bf16"), q, expert=torch.from_numpy(expert).cuda())["out"]
    torch.cuda.synchronize()
    W, A = ref.q4_decode(codes, moe_inputs.bits_to_f64(scale, "bf16"), z, (E, N, K), group, kind)
    got, x = bits_to_f64(to_host(out, "bf16"), "bf16"), bits_to_f64(host, "bf16")
    for r in range(R):
        want = W[expert[r]] @ x[r]
        bound = ref.STEP["bf16"] * np.abs(want) + 1.01 * (K + 8) * ref.ACC * (A[expert[r]] @ np.abs(x[r]))
        assert (np.abs(got[r] - want) <= bound + 1e-30).all(), r
