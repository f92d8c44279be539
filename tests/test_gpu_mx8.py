"""8-bit matrices (quantiser and way back) and the norm in front of the layer
with its gradient, against 64 bits, on the GPU."""
import copy

import numpy as np
import pytest

import routing_dispatch_expert_amd as moe
from tests import mx8_reference as ref
from tests.gpu_util import U, gpu_available, say

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}   # half a step, relative


@pytest.fixture(autouse=True)
def _gpu():
    assert gpu_available(), "GPU tests need an MI355X; run them with -m gpu on a GPU host"
    moe.lib()


def dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(DT[dtype]).cuda()


def host(t):
    return t.double().cpu().numpy()


def check_quantized(W, dtype):
    w = host(W)
    q = moe.quantize_mx8(W)
    K = w.shape[-1]
    bytes_ = ref.scale_bytes(w)
    assert np.array_equal(q.scale.cpu().numpy(), ref.pack_scale(bytes_, K))
    want = ref.values(w)
    codes = ref.decode(q.codes.view(torch.uint8).cpu().numpy())
    np.testing.assert_array_equal(codes * ref.two(ref.spread(bytes_, K)), want)
    for out in ("bf16", "f32"):
        np.testing.assert_array_equal(host(moe.dequantize_mx8(q, DT[out])), host(torch.from_numpy(want).to(DT[out])))
    return q


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 16), (3, 48), (1, 1, 128), (5, 33, 144), (2, 16, 256), (1, 1000, 1424), (70, 7168), (3, 7, 4112)])
def test_quantize(shape, dtype):
    say("quantize", shape, dtype)
    rng = np.random.default_rng(sum(shape))
    w = rng.standard_normal(shape) * np.exp(3 * rng.standard_normal((*shape[:-1], 1)))
    check_quantized(dev(w, dtype), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_at_the_edges(dtype):
    """Largest values around 448 times a power of two, ties between codes, small and huge groups, zeros."""
    rng = np.random.default_rng(2)
    w = np.zeros((12, 128), np.float32)
    w[0, ::32] = (448, 449 if dtype == "f32" else 450, 447, -448)
    w[1, ::32] = (np.nextafter(np.float32(448), 500), 1.75, 1.7500001, -0.875)
    w[2] = rng.integers(0, 113, 128) / 2 + 0.25 * rng.integers(0, 2, 128)
    w[3] = np.arange(128) * 2.0 ** -10          # subnormal codes and their ties
    w[3, ::32] = 300
    w[4] = 3e38 * rng.uniform(-1, 1, 128)
    w[5] = 1e-37 * rng.uniform(-1, 1, 128)
    w[6] = 1e-39 * rng.uniform(-1, 1, 128)      # below the smallest scale's reach
    w[7] = -0.0
    w[8, :32] = 0
    w[8, 32:] = rng.standard_normal(96)
    check_quantized(dev(w, dtype), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinities_and_nan_make_their_group_nan(dtype):
    w = np.random.default_rng(3).standard_normal((4, 160)).astype(np.float32)
    w[0, 5], w[1, 40], w[2, 159], w[2, 0] = np.nan, np.inf, -np.inf, -np.nan
    got = host(moe.dequantize_mx8(moe.quantize_mx8(dev(w, dtype)), DT["f32"]))
    bad = ref.spread(~np.isfinite(w.reshape(4, 5, 32)).all(-1), 160)
    assert np.isnan(got[bad]).all() and np.isfinite(got[~bad]).all()


def test_handles():
    W = torch.randn(3, 20, 64, device="cuda")
    q = moe.quantize_mx8(W)
    again = moe.Mx8(q.codes, q.scale)
    for other in (again, copy.deepcopy(q)):
        assert other.shape == (3, 20, 64) and torch.equal(moe.dequantize_mx8(other, torch.float32), moe.dequantize_mx8(q, torch.float32))
    with pytest.raises(AttributeError):
        q.codes = q.codes
    for bad in ((q.codes, q.scale[:, :, :19]), (q.codes.float(), q.scale), (q.codes[0], q.scale), (q.codes.view(torch.uint8), q.scale),
                (q.codes.transpose(1, 2), q.scale), (q.codes.cpu(), q.scale)):
        with pytest.raises((ValueError, moe.MoeError)):   # the last but one has 20 columns, which no 8-bit matrix has
            moe.Mx8(*bad)
    e = moe.quantize_mx8(torch.zeros(0, 64, device="cuda"))
    assert moe.dequantize_mx8(e, torch.bfloat16).shape == (0, 64)


# ------------------------------------------------------------------ the norm

def rows(rng, R, d, dtype):
    return dev(rng.standard_normal((R, d)) * np.exp(0.7 * rng.standard_normal(d)), dtype)


def depth(d, dtype):
    """Most roundings in a chain of a row's sum: a thread's elements (64 at most), six levels of lanes, sixteen waves."""
    return min(d, 64) + 6 + 16


NORMS = {"bf16": [(1, 16), (5, 48), (3, 512), (2, 1008), (70, 2048), (3, 2064), (2, 4096), (1, 7168), (9, 8208), (2, 16384), (2, 16400),
                  (1, 40000), (1, 65536)],
         "f32": [(1, 16), (3, 256), (2, 512), (70, 1024), (2, 1040), (3, 2048), (5, 4112), (1, 8192), (2, 8208), (1, 32768)]}


@pytest.mark.parametrize("dtype,R,d", [(t, *s) for t in NORMS for s in NORMS[t]])
def test_norm(dtype, R, d):
    rng = np.random.default_rng(R + d)
    x, res, w = rows(rng, R, d, dtype), rows(rng, R, d, dtype), dev(1 + 0.2 * rng.standard_normal(d), dtype)
    for residual in (None, res):
        say("norm", dtype, R, d, residual is not None)
        r = moe.rmsnorm(x, w, eps=1e-5, residual=residual, mx8=True)
        h = x if residual is None else (x.float() + residual.float()).to(DT[dtype])   # one rounding of an exact sum's fp32
        assert torch.equal(r["h"], h)
        v = host(h)
        rstd = 1 / np.sqrt((v * v).mean(1) + np.float64(np.float32(1e-5)))
        off = U * (depth(d, dtype) / 2 + 4)      # half of the sum's, and of the division, eps, root, reciprocal
        assert np.all(np.abs(host(r["rstd"]) - rstd) <= off * rstd)
        y = v * rstd[:, None] * host(w)
        off = (off + 2 * U) * np.abs(y)          # two products
        assert np.all(np.abs(host(r["y"]) - y) <= off + HALF[dtype] * (np.abs(y) + off))
        # 8 bits: the scale is right unless the group's largest lies within its error of 448 times a power of two; the
        # value is within half a step of the kernel's own y
        got = ref.unpack_scale(r["y8"].scale.cpu().numpy(), d)
        lo, hi = ref.scale_bytes(y * (1 - 2.0 ** -16)), ref.scale_bytes(y * (1 + 2.0 ** -16))
        assert np.all((lo <= got) & (got <= hi))
        s = ref.two(ref.spread(got, d))
        codes = ref.decode(r["y8"].codes.view(torch.uint8).cpu().numpy())
        assert np.all(np.abs(codes * s - y) <= off + s * ref.half_step(np.minimum(np.abs(y / s) * (1 + 2.0 ** -16), 448)))


def test_norm_outputs_asked_for():
    rng = np.random.default_rng(1)
    for dtype in DT:
        x, w = rows(rng, 6, 96, dtype), dev(1 + 0.2 * rng.standard_normal(96), dtype)
        a = moe.rmsnorm(x, w, mx8=True)
        b = moe.rmsnorm(x, w)
        c = moe.rmsnorm(x, w, want_y=False, mx8=True)
        assert torch.equal(a["y"], b["y"]) and b["y8"] is None and c["y"] is None and a["h"] is x
        assert torch.equal(a["y8"].codes.view(torch.uint8), c["y8"].codes.view(torch.uint8)) and torch.equal(a["y8"].scale, c["y8"].scale)
        n = x.shape[1]
        x4 = rows(rng, 3, 20 if dtype == "f32" else 24, dtype)   # widths that have no 8-bit form
        assert moe.rmsnorm(x4, torch.ones_like(x4[0]))["y"].shape == x4.shape
        with pytest.raises(moe.MoeError):
            moe.rmsnorm(x4, torch.ones_like(x4[0]), mx8=True)
        d = moe.rmsnorm(x, w, mx8=True, out=a)
        assert d is a
        with pytest.raises(ValueError):
            moe.rmsnorm(x, w, out=a)
        e = moe.rmsnorm(x[:0], w, residual=x[:0], mx8=True)
        assert e["y"].shape == (0, n) and e["y8"].shape == (0, n)


def test_norm_of_rows_of_zeros_and_with_infinities():
    for dtype in DT:
        x = torch.ones(5, 64, dtype=DT[dtype], device="cuda")
        x[0] = 0
        x[1, 3] = float("inf")
        x[2, 40] = float("nan")
        x[3] = 0
        r = moe.rmsnorm(x, torch.ones(64, dtype=DT[dtype], device="cuda"), eps=1e-6, mx8=True)
        v = moe.dequantize_mx8(r["y8"], torch.float32)
        eps = np.float64(np.float32(1e-6))
        # root and reciprocal: a step each, and one for eps + the mean of the last row
        assert not r["y"][0].any() and not v[0].any() and abs(r["rstd"][0].item() * eps ** 0.5 - 1) <= 4 * U
        assert r["y"][1, :3].eq(0).all() and r["y"][1, 3].isnan() and v[1, :32].isnan().all() and v[1, 32:].eq(0).all()
        assert r["y"][2].isnan().all() and v[2].isnan().all()
        one = (1 + eps) ** -0.5   # 1 in bf16 and in 8 bits
        assert np.all(np.abs(host(r["y"][4]) - one) <= 6 * U + HALF[dtype]) and (v[4] == 1).all()


BACK = {"bf16": [(1, 16), (5, 48), (3, 2048), (2500, 64), (300, 2064), (1100, 4096), (9, 8208), (3, 16400), (2, 65536)],
        "f32": [(1, 4), (1003, 500), (9, 1024), (30, 1040), (5, 8192), (300, 8208), (1, 32768)]}


@pytest.mark.parametrize("dtype,R,d", [(t, *s) for t in BACK for s in BACK[t]])
def test_norm_backward(dtype, R, d):
    rng = np.random.default_rng(R + d)
    h, w = rows(rng, R, d, dtype), dev(1 + 0.2 * rng.standard_normal(d), dtype)
    dy, dres = dev(rng.standard_normal((R, d)), dtype), dev(rng.standard_normal((R, d)), dtype)
    rstd = moe.rmsnorm(h, w)["rstd"]
    v, g, r = host(h), host(dy), host(rstd)[:, None]
    a, n = g * host(w), v * r
    steps = depth(d, dtype) + 8
    for extra in (None, dres):
        say("norm backward", dtype, R, d, extra is not None)
        res = moe.rmsnorm_backward(dy, h, w, rstd, dh=extra)
        e = 0 if extra is None else host(extra)
        want = r * (a - n * (a * n).mean(1, keepdims=True)) + e
        size = r * (np.abs(a) + np.abs(n) * np.abs(a * n).mean(1, keepdims=True)) + np.abs(e)
        off = U * steps * size
        assert np.all(np.abs(host(res["dh"]) - want) <= off + HALF[dtype] * (np.abs(want) + off))
        # of 256 to 2048 shares each adds up its rows, the last kernel a sixteenth of the shares and sixteen of those
        off = U * (R / 256 + 2048 / 16 + 16 + 4) * np.abs(g * n).sum(0)
        want = (g * n).sum(0)
        assert np.all(np.abs(host(res["dweight"]) - want) <= off + HALF[dtype] * (np.abs(want) + off))


def test_norm_backward_against_differences():
    rng = np.random.default_rng(4)
    h, w, dy = (rng.standard_normal(s) for s in ((2, 32), (32,), (2, 32)))
    hd, wd = dev(h, "f32"), dev(w, "f32")
    res = moe.rmsnorm_backward(dev(dy, "f32"), hd, wd, moe.rmsnorm(hd, wd, eps=1e-3)["rstd"])
    h, w, dy = (host(t) for t in (hd, wd, dev(dy, "f32")))
    loss = lambda h, w: (dy * h / np.sqrt((h * h).mean(1, keepdims=True) + np.float64(np.float32(1e-3))) * w).sum()  # noqa: E731
    step = 1e-5   # a central difference is off by step^2 times a third derivative of order 1 and by 2^-53 / step
    for at in np.ndindex(2, 32):
        e = np.zeros((2, 32))
        e[at] = step
        assert abs((loss(h + e, w) - loss(h - e, w)) / (2 * step) - host(res["dh"])[at]) < 1e-5
    for c in range(32):
        e = np.zeros(32)
        e[c] = step
        assert abs((loss(h, w + e) - loss(h, w - e)) / (2 * step) - host(res["dweight"])[c]) < 1e-5


def test_norm_backward_of_no_rows_and_in_place():
    for dtype in DT:
        z = torch.zeros(0, 64, dtype=DT[dtype], device="cuda")
        w = torch.ones(64, dtype=DT[dtype], device="cuda")
        r = moe.rmsnorm_backward(z, z, w, torch.zeros(0, device="cuda"))
        assert r["dh"].shape == (0, 64) and r["dweight"].eq(0).all()
    rng = np.random.default_rng(8)
    x, res, w, dy = (rows(rng, 40, 512, "bf16") for _ in range(4))
    w = w[0].contiguous()
    want = moe.rmsnorm(x, w, residual=res)
    y, rstd = torch.empty_like(x), torch.empty(40, device="cuda")
    moe.moe_rmsnorm(x, res, w, 1e-6, 40, 512, "bf16", res, y, None, rstd, torch.cuda.current_stream())   # the stream updated in place
    assert torch.equal(res, want["h"]) and torch.equal(y, want["y"]) and torch.equal(rstd, want["rstd"])
    back = moe.rmsnorm_backward(dy, res, w, rstd, dh=x)
    n = moe.moe_rmsnorm_backward_workspace_size(40, 512, "bf16")
    dw, ws = torch.empty_like(w), torch.empty(n, dtype=torch.uint8, device="cuda")
    moe.moe_rmsnorm_backward(dy, res, w, rstd, x, 40, 512, "bf16", x, dw, ws, n, torch.cuda.current_stream())
    assert torch.equal(x, back["dh"]) and torch.equal(dw, back["dweight"])
