"""Refusals and sizes of the 8-bit matrices' and the norm's entry points, on
the host: every call fails its checks before any GPU work."""
import numpy as np
import pytest

import routing_dispatch_expert_amd as moe
from tests import mx8_reference as ref

FAKE = 1 << 40   # never dereferenced
INVALID, UNSUPPORTED, WORKSPACE = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE


def refused(status, call):
    with pytest.raises(moe.MoeError) as ei:
        call()
    assert ei.value.status == status and moe.moe_last_error()


def convert(fn, **kw):
    a = dict(E=2, N=16, K=64, dtype="bf16", W=FAKE, q=(FAKE, FAKE))
    a.update(kw)
    if fn is moe.moe_mx8_quantize:
        fn(a["W"], a["E"], a["N"], a["K"], a["dtype"], a["q"])
    else:
        fn(a["q"], a["E"], a["N"], a["K"], a["dtype"], a["W"])


@pytest.mark.parametrize("fn", [moe.moe_mx8_quantize, moe.moe_mx8_dequantize])
@pytest.mark.parametrize("kw,status", [
    (dict(E=0), INVALID), (dict(N=-1), INVALID), (dict(K=0), INVALID), (dict(K=24), UNSUPPORTED), (dict(dtype=3), INVALID),
    (dict(W=None), INVALID), (dict(W=FAKE + 8), INVALID), (dict(q=None), INVALID), (dict(q=(None, FAKE)), INVALID),
    (dict(q=(FAKE, None)), INVALID), (dict(q=(FAKE + 8, FAKE)), INVALID), (dict(q=(FAKE, FAKE + 4)), INVALID),
    (dict(N=1 << 31), UNSUPPORTED), (dict(K=1 << 31), UNSUPPORTED), (dict(N=1 << 20, K=1 << 20), UNSUPPORTED),
    (dict(E=(1 << 26) - 4, N=1, K=16), UNSUPPORTED), (dict(E=1, N=((1 << 26) - 4) * 8, K=16), UNSUPPORTED)])
def test_conversions(fn, kw, status):
    refused(status, lambda: convert(fn, **kw))


def test_sizes():
    assert moe.moe_mx8_size(3, 10, 144) == (3 * 10 * 144, 3 * 2 * 10 * 4)
    assert moe.moe_mx8_size((1 << 26) - 5, 8, 128)[0] == ((1 << 26) - 5) * 1024
    assert moe.moe_mx8_size(1, 0, 16) == (0, 0)
    refused(UNSUPPORTED, lambda: moe.moe_mx8_size(1, 8, 40))


def norm(**kw):
    a = dict(x=FAKE, residual=FAKE * 2, weight=FAKE * 3, eps=1e-6, R=4, d=64, dtype="bf16", h_out=FAKE * 4, y=FAKE * 5,
             y8=(FAKE * 6, FAKE * 7), rstd=FAKE * 8)
    a.update(kw)
    moe.moe_rmsnorm(**a)


@pytest.mark.parametrize("kw,status", [
    (dict(R=-1), INVALID), (dict(d=0), INVALID), (dict(d=60), UNSUPPORTED), (dict(d=56), UNSUPPORTED), (dict(d=65552), UNSUPPORTED),
    (dict(dtype="f32", d=32784), UNSUPPORTED), (dict(dtype=9), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(x=None), INVALID), (dict(weight=None), INVALID), (dict(residual=None), INVALID), (dict(y8=(FAKE, None)), INVALID),
    (dict(x=FAKE + 8), INVALID), (dict(residual=FAKE * 2 + 8), INVALID), (dict(weight=FAKE * 3 + 2), INVALID),
    (dict(h_out=FAKE * 4 + 8), INVALID), (dict(y=FAKE * 5 + 8), INVALID), (dict(y8=(FAKE + 4, FAKE)), INVALID),
    (dict(h_out=FAKE + 128), INVALID), (dict(h_out=FAKE * 2 + 128), INVALID), (dict(y=FAKE), INVALID), (dict(y=FAKE * 2), INVALID),
    (dict(y=FAKE * 4), INVALID), (dict(R=1 << 26), UNSUPPORTED), (dict(R=1 << 24, d=4096), UNSUPPORTED),
    (dict(R=1 << 22, d=32768), UNSUPPORTED)])
def test_norm_refusals(kw, status):
    refused(status, lambda: norm(**kw))


def test_norm_of_no_rows():
    norm(R=0, x=None, residual=FAKE, weight=None, h_out=None, y=None, y8=None, rstd=None)


def back(**kw):
    a = dict(dy=FAKE, h=FAKE * 2, weight=FAKE * 3, rstd=FAKE * 4, dh_in=FAKE * 5, R=4, d=64, dtype="bf16", dh=FAKE * 6,
             dweight=FAKE * 7, workspace=FAKE * 8, workspace_bytes=1 << 30)
    a.update(kw)
    moe.moe_rmsnorm_backward(**a)


@pytest.mark.parametrize("kw,status", [
    (dict(R=-1), INVALID), (dict(d=0), INVALID), (dict(d=60), UNSUPPORTED), (dict(d=65544), UNSUPPORTED), (dict(dtype=9), INVALID),
    (dict(dy=None), INVALID), (dict(h=None), INVALID), (dict(weight=None), INVALID), (dict(rstd=None), INVALID), (dict(dh=None), INVALID),
    (dict(dweight=None), INVALID), (dict(dy=FAKE + 8), INVALID), (dict(dh=FAKE * 6 + 8), INVALID), (dict(dh=FAKE + 128), INVALID),
    (dict(dh=FAKE * 2 + 128), INVALID), (dict(dh=FAKE * 5 + 128), INVALID), (dict(workspace=None), WORKSPACE),
    (dict(workspace_bytes=255), WORKSPACE), (dict(workspace=FAKE * 8 + 128), WORKSPACE), (dict(R=1 << 26), UNSUPPORTED)])
def test_norm_backward_refusals(kw, status):
    refused(status, lambda: back(**kw))


def test_the_reference_itself():
    assert ref.scale_bytes(np.array([[448.0] * 32 + [449.0] + [0.0] * 31 + [0.0] * 16])).tolist() == [[127, 128, 127]]
    every = ref.decode(np.arange(256))
    finite = every[np.isfinite(every)]
    assert finite.max() == 448 and len(finite) == 254
    w = finite[None]
    assert np.array_equal(ref.values(np.concatenate([w, [[0.0, 448.0]]], 1))[:, 224:254], w[:, 224:])
