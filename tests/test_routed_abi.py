"""Refusals of the layer with a given routing, on the host: every call fails its checks before any GPU work."""
import pytest

import routing_dispatch_expert_amd as moe

FAKE = 1 << 40   # never dereferenced
INVALID, UNSUPPORTED, WORKSPACE = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE


def forward(**kw):
    a = dict(x=FAKE, residual=FAKE * 2, topk_idx=FAKE, topk_w=FAKE, W_gate=FAKE, W_up=FAKE, W_down=FAKE, T=8, d=128, d_ff=64, E=8, k=2,
             cf=1.25, P=1, dtype="bf16", out=FAKE * 3, stats=None, workspace=FAKE * 4, workspace_bytes=1 << 40)
    a.update(kw)
    moe.moe_layer_forward_routed(**a)


def backward(**kw):
    a = dict(x=FAKE, topk_idx=FAKE, topk_w=FAKE, W_gate=FAKE, W_up=FAKE, W_down=FAKE, dout=FAKE * 2, T=8, d=128, d_ff=64, E=8, k=2,
             cf=1.25, P=1, dtype="bf16", saved=None, dx=FAKE * 3, d_topk_w=FAKE, dW_gate=FAKE, dW_up=FAKE, dW_down=FAKE,
             workspace=FAKE * 4, workspace_bytes=1 << 40)
    a.update(kw)
    moe.moe_layer_backward_routed(**a)


BOTH = [(dict(k=0), INVALID), (dict(k=9), INVALID), (dict(E=0), INVALID), (dict(T=-1), INVALID), (dict(cf=0.0), INVALID),
        (dict(P=3), INVALID), (dict(d=0), INVALID), (dict(dtype=5), INVALID), (dict(d=12), UNSUPPORTED), (dict(E=8192), UNSUPPORTED),
        (dict(E=64, k=33), UNSUPPORTED), (dict(x=None), INVALID), (dict(topk_idx=None), INVALID), (dict(topk_w=None), INVALID),
        (dict(W_gate=None), INVALID), (dict(W_up=None), INVALID), (dict(W_down=None), INVALID), (dict(workspace=None), WORKSPACE),
        (dict(workspace_bytes=100), WORKSPACE), (dict(workspace=FAKE * 4 + 8), WORKSPACE)]


@pytest.mark.parametrize("kw,status", BOTH)
@pytest.mark.parametrize("fn", [forward, backward])
def test_refusals(fn, kw, status):
    with pytest.raises(moe.MoeError) as ei:
        fn(**kw)
    assert ei.value.status == status and moe.moe_last_error()


@pytest.mark.parametrize("fn,kw", [
    (forward, dict(residual=None)), (forward, dict(out=None)), (forward, dict(out=FAKE + 64)), (forward, dict(out=FAKE * 2 + 64)),
    (forward, dict(stats=dict(topk_idx=FAKE))), (forward, dict(stats=dict(topk_w=FAKE))), (backward, dict(dout=None)),
    (backward, dict(dx=None)), (backward, dict(d_topk_w=None)), (backward, dict(dW_up=None)), (backward, dict(dx=FAKE + 64)),
    (backward, dict(dx=FAKE * 2 + 64)), (backward, dict(saved=dict(buckets=FAKE, g=FAKE, u=FAKE))),
    (backward, dict(saved=dict(g=FAKE, u=FAKE, h=FAKE)))])
def test_pointers(fn, kw):
    with pytest.raises(moe.MoeError) as ei:
        fn(**kw)
    assert ei.value.status == INVALID


def test_no_tokens():
    forward(T=0)
    backward(T=0)
