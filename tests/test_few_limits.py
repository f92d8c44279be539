"""Empty batches and the largest sizes of the few-token layer and the 4-bit weights, on the host: what is refused and
what passes its checks."""
import pytest

import routing_dispatch_expert_amd as moe
from tests.test_few_abi import FAKE, INVALID, _few, q4, refused


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
