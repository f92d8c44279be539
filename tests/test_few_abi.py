"""Refusals and sizes of the few-token layer's and the 4-bit weights' entry
points, on the host: every call fails its checks before any GPU work."""
import ctypes

import numpy as np
import pytest

import routing_dispatch_expert_amd as moe
from tests import few_reference as ref

FAKE = 1 << 40   # never dereferenced
INVALID, UNSUPPORTED, WORKSPACE = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE
STATS = {n: FAKE for n in ("topk_idx", "topk_w", "slot", "routed_count", "kept_count", "send_count", "totals")}


def q4(**kw):
    a = dict(codes=FAKE, scale=FAKE, zero=FAKE, kind="u4", group=64)
    a.update(kw)
    return a["codes"], a["scale"], a["zero"], a["kind"], a["group"]


def _few(fn, w, **kw):
    a = dict(x=FAKE, W_router=FAKE, router_bias=None, W_gate=w, W_up=w, W_down=w, T=8, d=128, d_ff=256, E=8, k=2, cf=1.25,
             P=1, max_ranks=0, dtype="bf16", out=FAKE * 2, stats=STATS, workspace=FAKE * 3, workspace_bytes=1 << 40,
             stream=None)
    a.update(kw)
    return fn(**a)


def refused(status, call):
    with pytest.raises(moe.MoeError) as ei:
        call()
    assert ei.value.status == status
    assert moe.moe_last_error()


LAYER = [
    (dict(k=0), INVALID), (dict(k=9), INVALID), (dict(E=0), INVALID), (dict(T=-1), INVALID), (dict(cf=0.0), INVALID),
    (dict(cf=float("nan")), INVALID), (dict(cf=float("inf")), INVALID), (dict(P=3), INVALID), (dict(P=0), INVALID),
    (dict(d=0), INVALID), (dict(d_ff=0), INVALID), (dict(dtype=5), INVALID), (dict(x=None), INVALID),
    (dict(W_router=None), INVALID), (dict(W_gate=None), INVALID), (dict(W_up=None), INVALID), (dict(W_down=None), INVALID),
    (dict(out=None), INVALID), (dict(out=FAKE + 64), INVALID), (dict(x=FAKE + 8), INVALID),
    (dict(W_router=FAKE + 4), INVALID), (dict(out=FAKE * 2 + 2), INVALID), (dict(max_ranks=-1), INVALID),
    (dict(E=8, k=4, P=4, max_ranks=1), INVALID), (dict(E=256, k=8, P=128, max_ranks=4), UNSUPPORTED),
    (dict(T=65), UNSUPPORTED), (dict(T=1 << 40), UNSUPPORTED), (dict(E=1025), UNSUPPORTED),
    (dict(E=64, k=33), UNSUPPORTED), (dict(d=12), UNSUPPORTED), (dict(d_ff=100), UNSUPPORTED),
    (dict(d=1 << 20, d_ff=1 << 20), UNSUPPORTED), (dict(d=(1 << 22) + 8, d_ff=8), UNSUPPORTED),
    (dict(d_ff=(1 << 22) + 8, d=8), UNSUPPORTED), (dict(workspace=None), WORKSPACE),
    (dict(E=1024, k=4, T=64, d=8, d_ff=1 << 22), UNSUPPORTED), (dict(workspace_bytes=100), WORKSPACE), (dict(workspace=FAKE * 3 + 8), WORKSPACE),
    (dict(stats=dict(STATS, buckets=FAKE)), INVALID), (dict(stats=dict(STATS, src=FAKE)), INVALID),
    (dict(stats=dict(STATS, instance=FAKE)), INVALID), (dict(stats=dict(STATS, g=FAKE, u=FAKE, h=FAKE)), INVALID),
]


@pytest.mark.parametrize("kw,status", LAYER)
def test_few_layer_refusals(kw, status):
    refused(status, lambda: _few(moe.moe_layer_forward_few, FAKE, **kw))
    refused(status, lambda: _few(moe.moe_layer_forward_few_q4, q4(), **kw))


def test_few_layer_refuses_misaligned_weights():
    for n in ("W_gate", "W_up", "W_down"):
        refused(INVALID, lambda: _few(moe.moe_layer_forward_few, FAKE, **{n: FAKE + 8}))


@pytest.mark.parametrize("bad", [dict(kind=2), dict(kind=-1), dict(group=16), dict(group=0), dict(codes=None),
                                 dict(scale=None), dict(codes=FAKE + 8), dict(scale=FAKE + 2), dict(zero=FAKE + 1),
                                 dict(kind="e2m1"), dict(group=32), dict(zero=None)], ids=str)
def test_few_layer_q4_refuses_bad_or_differing_weights(bad):
    for n in ("W_gate", "W_up", "W_down"):
        refused(INVALID, lambda: _few(moe.moe_layer_forward_few_q4, q4(), **{n: q4(**bad)}))


def test_fp32_widths():
    _few(moe.moe_layer_forward_few, FAKE, T=0, dtype="f32", d=132, d_ff=100)
    refused(UNSUPPORTED, lambda: _few(moe.moe_layer_forward_few, FAKE, dtype="f32", d=130))
    # 4-bit words hold eight columns
    refused(UNSUPPORTED, lambda: _few(moe.moe_layer_forward_few_q4, q4(), dtype="f32", d=132))
    refused(UNSUPPORTED, lambda: _few(moe.moe_layer_forward_few_q4, q4(), dtype="f32", d_ff=100))


def test_nothing_to_do():
    _few(moe.moe_layer_forward_few, FAKE, T=0, workspace=None, workspace_bytes=0)
    _few(moe.moe_layer_forward_few_q4, q4(), T=0, workspace=None, workspace_bytes=0, stats=None)
    assert moe.moe_few_workspace_size(0, 128, 256, 8, 2, 1.25, 1, "bf16", 0) >= 0
    moe.moe_q4_matvec(FAKE, None, q4(), 0, 1, 16, 128, "bf16", FAKE * 2, None, 0)


def test_few_workspace_size():
    size = moe.moe_few_workspace_size
    a = size(1, 7168, 2048, 256, 8, 2.0, 8, "bf16", 0)
    assert a >= 8 * 2048 * 2            # h of eight copies
    assert size(64, 7168, 2048, 256, 8, 2.0, 8, "bf16", 0) > a
    assert size(1, 7168, 2048, 256, 8, 2.0, 8, "f32", 1) > a   # three parts of x and h
    for bad, status in ((dict(T=65), UNSUPPORTED), (dict(E=1032), UNSUPPORTED), (dict(k=0), INVALID)):
        k = dict(T=1, d=128, d_ff=256, E=8, k=2, cf=1.0, P=1, dtype="bf16", q4=0)
        k.update(bad)
        refused(status, lambda: size(**k))
    assert moe.lib().moe_few_workspace_size(1, 128, 256, 8, 2, 1.0, 1, 1, 0, None) == INVALID


@pytest.mark.parametrize("E,N,K,group", [(1, 1, 8, 32), (3, 17, 136, 64), (4, 128, 256, 128), (256, 2048, 7168, 128)])
def test_q4_size(E, N, K, group):
    cs, ss = ref.q4_shapes(E, N, K, group)
    assert moe.moe_q4_size(E, N, K, group) == (int(np.prod(cs)), 2 * int(np.prod(ss)), int(np.prod(ss)))
    n = ctypes.c_size_t(0)
    assert moe.lib().moe_q4_size(E, N, K, group, None, ctypes.byref(n), None) == moe.MOE_OK
    assert n.value == 2 * int(np.prod(ss))


SHAPES = [(dict(E=0), INVALID), (dict(N=0), INVALID), (dict(K=-8), INVALID), (dict(K=12), UNSUPPORTED),
          (dict(N=1 << 40), UNSUPPORTED), (dict(E=1 << 16, N=1 << 16, K=1 << 12), UNSUPPORTED),
          (dict(E=1 << 12, N=1 << 14, K=1 << 11), UNSUPPORTED)]


@pytest.mark.parametrize("kw,status", SHAPES)
def test_q4_shape_refusals(kw, status):
    a = dict(E=2, N=32, K=128)
    a.update(kw)
    refused(status, lambda: moe.moe_q4_size(*a.values(), 64))
    refused(status, lambda: moe.moe_q4_quantize(FAKE, *a.values(), "bf16", q4()))
    refused(status, lambda: moe.moe_q4_dequantize(q4(), *a.values(), "bf16", FAKE))
    refused(status, lambda: moe.moe_q4_matvec(FAKE, None, q4(), 4, *a.values(), "bf16", FAKE * 2, None, 0))


@pytest.mark.parametrize("bad", [dict(kind=2), dict(group=48), dict(codes=None), dict(scale=None), dict(codes=FAKE + 4),
                                 dict(kind="e2m1")], ids=str)
def test_q4_weight_refusals(bad):
    refused(INVALID, lambda: moe.moe_q4_quantize(FAKE, 2, 32, 128, "bf16", q4(**bad)))
    refused(INVALID, lambda: moe.moe_q4_dequantize(q4(**bad), 2, 32, 128, "bf16", FAKE))
    refused(INVALID, lambda: moe.moe_q4_matvec(FAKE, None, q4(**bad), 4, 2, 32, 128, "bf16", FAKE * 2, None, 0))


def test_largest_q4_sizes():
    assert moe.moe_q4_size((1 << 12) - 1, 1 << 14, 1 << 11, 64)[0] == ((1 << 12) - 1) << 24


def test_q4_argument_refusals():
    refused(INVALID, lambda: moe.moe_q4_quantize(None, 2, 32, 128, "bf16", q4()))
    refused(INVALID, lambda: moe.moe_q4_quantize(FAKE + 8, 2, 32, 128, "bf16", q4()))
    refused(INVALID, lambda: moe.moe_q4_quantize(FAKE, 2, 32, 128, 7, q4()))
    refused(INVALID, lambda: moe.moe_q4_quantize(FAKE, 2, 32, 128, "bf16", None))
    refused(INVALID, lambda: moe.moe_q4_dequantize(q4(), 2, 32, 128, 7, FAKE))
    refused(INVALID, lambda: moe.moe_q4_dequantize(q4(), 2, 32, 128, "bf16", None))
    mv = moe.moe_q4_matvec
    refused(INVALID, lambda: mv(None, None, q4(), 4, 2, 32, 128, "bf16", FAKE * 2, None, 0))
    refused(INVALID, lambda: mv(FAKE, None, q4(), 4, 2, 32, 128, "bf16", None, None, 0))
    refused(INVALID, lambda: mv(FAKE, None, q4(), -1, 2, 32, 128, "bf16", FAKE * 2, None, 0))
    refused(INVALID, lambda: mv(FAKE, None, q4(), 4, 2, 32, 128, "bf16", FAKE + 64, None, 0))
    refused(INVALID, lambda: mv(FAKE + 2, None, q4(), 4, 2, 32, 128, "bf16", FAKE * 2, None, 0))
    refused(UNSUPPORTED, lambda: mv(FAKE, None, q4(), 4, 1, 8, (1 << 22) + 8, "bf16", FAKE << 10, None, 0))
    refused(UNSUPPORTED, lambda: mv(FAKE, None, q4(), 65, 2, 32, 128, "bf16", FAKE * 2, None, 0))
    refused(WORKSPACE, lambda: mv(FAKE, None, q4(), 4, 2, 32, 128, "f32", FAKE * 2, None, 0))
    refused(WORKSPACE, lambda: mv(FAKE, None, q4(), 4, 2, 32, 128, "f32", FAKE * 2, FAKE * 3 + 16, 1 << 30))
    size = moe.moe_q4_matvec_workspace_size
    assert size(64, 7168, "bf16") == 0 and size(3, 136, "f32") >= 3 * 136 * 6
    refused(INVALID, lambda: size(-1, 128, "f32"))
    refused(INVALID, lambda: size(1, 128, 9))
    assert moe.lib().moe_q4_matvec_workspace_size(1, 8, 0, None) == INVALID


def test_python_handles_refuse_what_does_not_fit():
    torch = pytest.importorskip("torch")
    cs, ss = ref.q4_shapes(2, 32, 256, 64)
    codes, scale = torch.zeros(cs, dtype=torch.uint8), torch.zeros(ss, dtype=torch.bfloat16)
    with pytest.raises(ValueError):   # host memory
        moe.Q4Weights(codes, scale, None, (2, 32, 256), 64, "u4")
    with pytest.raises(ValueError):
        moe.Q4Weights(codes, scale, None, (2, 32, 256), 64, "int4")
    with pytest.raises(moe.MoeError):
        moe.Q4Weights(codes, scale, None, (2, 32, 256), 48, "u4")
    with pytest.raises(ValueError):
        moe.quantize_q4(torch.zeros(32, 256))
    with pytest.raises(ValueError):
        moe.quantize_q4(torch.zeros(1, 32, 256))
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        moe.forward_few(x, torch.zeros(8, 64), *(torch.zeros(8, 64, 64) for _ in range(3)), k=2, cf=1.0)


def test_reference_layout_round_trip():
    """The reference's own codes decode to the nearest representable values (its two halves agree)."""
    rng = np.random.default_rng(2)
    w = rng.standard_normal((2, 21, 200)).astype(np.float32)
    for kind, zero in (("u4", True), ("u4", False), ("e2m1", False)):
        codes, s, z = ref.q4_quantize(w, 32, kind, zero)
        W, _ = ref.q4_decode(codes, s.astype(np.float64), z, w.shape, 32, kind)
        g = np.arange(200) // 32
        per = s.transpose(0, 1, 3, 2).reshape(2, 32, -1)[:, :21][:, :, g]
        # half of the widest step: 1 (u4), 2 (e2m1) scales; a clipped end of the range adds half a step, and a
        # scale that was rounded down cuts 2^-8 of the range's largest value
        assert (np.abs(W - w) <= per * (1.0 if kind != "u4" else 0.5 if not zero else 1.0) + np.abs(w) * 2.0 ** -7).all()
