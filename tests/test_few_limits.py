"""Empty batches and the largest sizes of the few-token layer and the 4-bit weights, on the host: what is refused and
what passes its checks."""
import pytest

import routing_dispatch_expert_amd as moe
from tests.test_few_abi import FAKE, INVALID, UNSUPPORTED, _few, q4, refused


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_tokens_need_no_addresses(dtype):
    """An empty tensor's address is NULL."""
    empty = dict(T=0, x=None, out=None, dtype=dtype, workspace=None, workspace_bytes=0)
    _few(moe.moe_layer_forward_few, FAKE, **empty)
    _few(moe.moe_layer_forward_few_q4, q4(), **empty)
    moe.moe_q4_matvec(None, None, q4(), 0, 4, 16, 128, dtype, None, None, 0)
    # the weights are still checked
    refused(INVALID, lambda: _few(moe.moe_layer_forward_few, FAKE, **dict(empty, W_router=None)))
    refused(INVALID, lambda: _few(moe.moe_layer_forward_few, None, **empty))
    refused(INVALID, lambda: moe.moe_q4_matvec(None, None, q4(codes=None), 0, 4, 16, 128, dtype, None, None, 0))
    for name in ("x", "out"):
        refused(INVALID, lambda: _few(moe.moe_layer_forward_few, FAKE, **{name: None}))
    for x, out in ((None, FAKE), (FAKE, None)):
        refused(INVALID, lambda: moe.moe_q4_matvec(x, None, q4(), 1, 4, 16, 128, dtype, out, FAKE * 3, 1 << 20))


@pytest.mark.parametrize("E,N,K", [(1, 16 * (2 ** 26 - 4), 8), (1, 16, 128 * (2 ** 24 - 1)), (2 ** 26 - 4, 1, 8),
                                   (4, 16 * (2 ** 24 - 1), 128), (3, 16 * ((2 ** 26 - 4) // 3), 8)])
def test_largest_stack_of_tiles(E, N, K):
    """The quantiser's launch takes 256 threads for four tiles: at most 2^26 - 4 of them stay below 2^32."""
    tiles = E * -(-N // 16) * -(-K // 128)
    assert tiles <= 2 ** 26 - 4 and 256 * -(-tiles // 4) < 2 ** 32
    assert moe.moe_q4_size(E, N, K, 32)[0] == tiles * 1024


@pytest.mark.parametrize("E,N,K", [(1, 16 * (2 ** 26 - 4) + 1, 8), (1, 16 * (2 ** 26 - 1), 8), (2 ** 26 - 3, 1, 8),
                                   (2 ** 26 - 1, 16, 128), (3, 16 * ((2 ** 26 - 4) // 3) + 1, 8), (1, 2 ** 30, 8)])
def test_one_tile_too_many(E, N, K):
    refused(UNSUPPORTED, lambda: moe.moe_q4_size(E, N, K, 32))
    q = q4(group=32, zero=None)
    refused(UNSUPPORTED, lambda: moe.moe_q4_quantize(FAKE, E, N, K, "bf16", q))
    refused(UNSUPPORTED, lambda: moe.moe_q4_dequantize(q, E, N, K, "bf16", FAKE))
    refused(UNSUPPORTED, lambda: moe.moe_q4_matvec(FAKE, None, q, 1, E, N, K, "bf16", FAKE * 2, None, 0))
