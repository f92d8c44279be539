"""Refusals of the 8-bit experts' entry points, on the host: every call fails its checks before any GPU work."""
import pytest

import routing_dispatch_expert_amd as moe

FAKE = 1 << 40   # never dereferenced
INVALID, UNSUPPORTED, WORKSPACE = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE
Q = (FAKE, FAKE * 2)


def call(**kw):
    a = dict(x=Q, residual=FAKE * 3, topk_idx=FAKE, topk_w=FAKE, W_gate=Q, W_up=Q, W_down=Q, T=8, d=128, d_ff=64, E=8, k=2, cf=1.25,
             dtype="bf16", out=FAKE * 4, stats=dict(slot=FAKE, routed_count=FAKE, kept_count=FAKE), workspace=FAKE * 5,
             workspace_bytes=1 << 40)
    a.update(kw)
    moe.moe_experts_mx8(**a)


SHAPES = [(dict(k=0), INVALID), (dict(k=9), INVALID), (dict(E=0), INVALID), (dict(T=-1), INVALID), (dict(cf=0.0), INVALID),
          (dict(cf=float("nan")), INVALID), (dict(d=0), INVALID), (dict(d_ff=0), INVALID), (dict(dtype=5), INVALID),
          (dict(d=136), UNSUPPORTED), (dict(d_ff=72), UNSUPPORTED), (dict(E=8192), UNSUPPORTED), (dict(E=64, k=33), UNSUPPORTED),
          (dict(d=1 << 16, d_ff=1 << 16), UNSUPPORTED), (dict(T=1 << 24, cf=0.01), UNSUPPORTED), (dict(T=1 << 22, d=16, d_ff=16, cf=0.01), UNSUPPORTED),
          (dict(E=4096, T=4096, d=1 << 15, d_ff=16), UNSUPPORTED), (dict(E=1, k=1, T=1, d=1 << 28, d_ff=16), UNSUPPORTED)]


@pytest.mark.parametrize("kw,status", SHAPES + [
    (dict(x=None), INVALID), (dict(x=(FAKE, None)), INVALID), (dict(x=(FAKE + 8, FAKE)), INVALID), (dict(residual=None), INVALID),
    (dict(topk_idx=None), INVALID), (dict(topk_w=None), INVALID), (dict(out=None), INVALID), (dict(W_gate=None), INVALID),
    (dict(W_up=(None, FAKE)), INVALID), (dict(W_down=(FAKE, FAKE + 4)), INVALID), (dict(residual=FAKE * 3 + 8), INVALID),
    (dict(out=FAKE * 4 + 2), INVALID), (dict(out=FAKE * 3 + 256), INVALID), (dict(workspace=None), WORKSPACE),
    (dict(workspace_bytes=100), WORKSPACE), (dict(workspace=FAKE * 5 + 128), WORKSPACE)]
    + [(dict(stats={n: FAKE}), INVALID) for n in ("topk_idx", "topk_w", "src", "send_count", "totals", "buckets", "instance", "g", "h")])
def test_refusals(kw, status):
    with pytest.raises(moe.MoeError) as ei:
        call(**kw)
    assert ei.value.status == status and moe.moe_last_error()


@pytest.mark.parametrize("kw,status", SHAPES)
def test_sizes_are_checked_alike(kw, status):
    a = dict(T=8, d=128, d_ff=64, E=8, k=2, cf=1.25, dtype="bf16")
    a.update(kw)
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_experts_mx8_workspace_size(**a)
    assert ei.value.status == status


def test_no_tokens():
    call(T=0, x=None, residual=None, topk_idx=None, topk_w=None, out=None, workspace=None)
