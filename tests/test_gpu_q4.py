"""4-bit weights on the GPU: quantising and reading back, bit for bit against
numpy in fp32, and products of rows with them against 64 bits."""
import numpy as np
import pytest

import moe_inputs
import routing_dispatch_expert_amd as moe
from tests import few_reference as ref
from tests.gpu_util import Guarded, bits_to_f64, gpu_available, say, to_dev, to_host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(autouse=True)
def _gpu():
    assert gpu_available(), "GPU tests need an MI355X; run them with -m gpu on a GPU host"
    moe.lib()


KINDS = [("u4", True), ("u4", False), ("e2m1", False)]


def _weights(rng, shape, dtype):
    """Gaussian weights with rows of zeros, constant groups, one-sided groups and large and tiny values."""
    w = rng.standard_normal(shape).astype(np.float32)
    E, N, K = shape
    w[0, 0] = 0
    w[-1, -1] = 0.75
    w[0, N // 2] = np.abs(w[0, N // 2])
    w[0, N // 3] = -np.abs(w[0, N // 3])
    w[:, :, K // 2] *= 1e4
    w[0, N - 1] *= 1e-20
    return moe_inputs.to_bf16_bits(w) if dtype == "bf16" else w


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind,zero", KINDS)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("shape", [(1, 1, 8), (2, 16, 128), (3, 37, 200), (1, 130, 1032), (5, 8, 136)])
def test_quantize_and_back(shape, group, kind, zero, dtype):
    say(f"quantize {dtype} {shape} {kind} {group} {zero}")
    E, N, K = shape
    host = _weights(np.random.default_rng(N + K), shape, dtype)
    W = to_dev(host, dtype)
    cs, ss = ref.q4_shapes(E, N, K, group)
    assert moe.moe_q4_size(E, N, K, group) == (int(np.prod(cs)), 2 * int(np.prod(ss)), int(np.prod(ss)))
    g = Guarded()
    codes = g.empty((int(np.prod(cs)) // 4,), torch.int32, "codes")
    scale = g.empty(ss, torch.bfloat16, "scale")
    zt = g.empty((int(np.prod(ss)) // 4,), torch.int32, "zero") if kind == "u4" and zero else None
    moe.moe_q4_quantize(W, E, N, K, dtype, (codes, scale, zt, kind, group))
    back = g.empty(shape, W.dtype, "values")
    moe.moe_q4_dequantize((codes, scale, zt, kind, group), E, N, K, dtype, back)
    torch.cuda.synchronize()
    g.check()
    want = ref.q4_quantize(bits_to_f64(host, dtype).astype(np.float32), group, kind, zero)
    s64 = moe_inputs.bits_to_f64(to_host(scale, "bf16"), "bf16")
    assert np.array_equal(s64, want[1]), "scale"
    z = None
    if zt is not None:
        z = zt.cpu().numpy().view(np.uint8).reshape(ss)
        assert np.array_equal(z, want[2]), "zero"
    c = codes.cpu().numpy().view(np.uint8).reshape(cs)
    have, _ = ref.q4_decode(c, s64, z, shape, group, kind)
    should, _ = ref.q4_decode(want[0], want[1].astype(np.float64), want[2], shape, group, kind)
    assert np.array_equal(have, should), "codes"
    got = bits_to_f64(to_host(back, dtype), dtype)
    rounded = bits_to_f64(moe_inputs.to_bf16_bits(have.astype(np.float32)), "bf16") if dtype == "bf16" else have
    assert np.array_equal(got, rounded), "values"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind,zero", KINDS)
def test_quantize_at_the_edges_between_codes(kind, zero, dtype):
    """Quotients on, and one unit beside, every edge between two codes, at scales from subnormal to the largest."""
    rng = np.random.default_rng(17)
    edges = np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6] if kind == "e2m1" else np.arange(.5, 15, 1), np.float32)
    top = np.float32(6 if kind == "e2m1" else 15 if zero else 7)
    rows = []
    for exp in (-140, -126, -120, -101, -100, -99, -60, -1, 0, 1, 60, 122, 124):
        for _ in range(4):
            s = np.float32(1 + rng.integers(0, 128) / 128) * np.float32(2.0) ** exp
            e = rng.choice(edges, 32) * (1 if kind == "u4" and zero else rng.choice([-1, 1], 32))
            v = (e.astype(np.float64) * np.float64(s)).astype(np.float32)
            v = np.nextafter(v, rng.choice([-np.inf, np.inf], 32).astype(np.float32), where=rng.random(32) < .5, out=v)
            v = np.clip(v, -top * s, top * s)
            v[3] = top * s
            rows.append(v)
    w = np.array(rows, np.float32)[None]
    host = moe_inputs.to_bf16_bits(w) if dtype == "bf16" else w
    q = moe.quantize_q4(to_dev(host, dtype), group=32, kind=kind, zero_points=zero)
    torch.cuda.synchronize()
    # 15 2^124 passes fp32's range: rows with infinities, which weights must not hold, are only quantised, not compared
    finite = np.isfinite(bits_to_f64(host, dtype)).all(-1)[0]
    assert finite[:48].all()
    want = ref.q4_quantize(bits_to_f64(host, dtype).astype(np.float32), 32, kind, zero)
    s64 = moe_inputs.bits_to_f64(to_host(q.scale, "bf16"), "bf16")
    row = np.pad(finite, (0, -len(finite) % 16)).reshape(1, -1, 1, 16) & np.ones(s64.shape, bool)
    assert np.array_equal(s64[row], want[1][row]), "scale"
    z = None if q.zero is None else q.zero.cpu().numpy()
    assert z is None or np.array_equal(z[row], want[2][row]), "zero"
    with np.errstate(invalid="ignore"):
        have, _ = ref.q4_decode(q.codes.cpu().numpy(), s64, z, w.shape, 32, kind)
        should, _ = ref.q4_decode(want[0], want[1].astype(np.float64), want[2], w.shape, 32, kind)
    assert np.array_equal(have[0, finite], should[0, finite]), "codes"


def test_quantizing_codes_values_again_keeps_them():
    """Values that 4 bits hold exactly come back unchanged."""
    rng = np.random.default_rng(3)
    w = torch.from_numpy(rng.choice(ref.E2M1[:8], (2, 32, 256)).astype(np.float32)).cuda()
    w[:, :, ::32] = 6.0
    assert torch.equal(moe.dequantize_q4(moe.quantize_q4(w, group=32, kind="e2m1"), torch.float32), w)
    v = torch.from_numpy(rng.integers(-8, 8, (2, 32, 256)).astype(np.float32)).cuda()
    v[:, :, 0], v[:, :, 128], v[:, :, 1], v[:, :, 129] = -8, -8, 7, 7
    assert torch.equal(moe.dequantize_q4(moe.quantize_q4(v, group=128), torch.float32), v)


MATVEC = [  # R, N, K, E
    (1, 1, 8, 1), (1, 40, 136, 1), (2, 130, 512, 3), (5, 24, 72, 2), (16, 64, 256, 1), (17, 48, 128, 1),
    (33, 33, 264, 4), (64, 16, 128, 64), (64, 100, 392, 1), (64, 56, 1160, 7),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind,zero", KINDS)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("R,N,K,E", MATVEC)
def test_matvec(R, N, K, E, group, kind, zero, dtype):
    say(f"matvec {dtype} R={R} N={N} K={K} E={E} {kind} {group} {zero}")
    rng = np.random.default_rng(R * 1000 + N)
    codes, scale, z = ref.random_q4(rng, E, N, K, group, kind, zero)
    host = rng.standard_normal((R, K)).astype(np.float32)
    host = moe_inputs.to_bf16_bits(host) if dtype == "bf16" else host
    expert = rng.integers(0, E, R).astype(np.int32)
    if R > 4:
        expert[[1, R - 1]] = [-1, E]   # rows without a matrix
    x = to_dev(host, dtype)
    q = moe.Q4Weights(torch.from_numpy(codes).cuda(), to_dev(scale, "bf16"),
                      None if z is None else torch.from_numpy(z).cuda(), (E, N, K), group, kind)
    g = Guarded()
    out = g.empty((R, N), x.dtype, "out")
    out.fill_(7.0)
    n = moe.moe_q4_matvec_workspace_size(R, K, dtype)
    ws = g.empty((n // 4,), torch.int32, "workspace")
    moe.moe_q4_matvec(x, torch.from_numpy(expert).cuda(), q, R, E, N, K, dtype, out, ws, n)
    torch.cuda.synchronize()
    g.check()
    W, A = ref.q4_decode(codes, moe_inputs.bits_to_f64(scale, "bf16"), z, (E, N, K), group, kind)
    x64 = bits_to_f64(host, dtype)
    got = bits_to_f64(to_host(out, dtype), dtype)
    for r in range(R):
        if not 0 <= expert[r] < E:
            assert (got[r] == 7).all(), f"row {r} has no matrix and was written"
            continue
        want = W[expert[r]] @ x64[r]
        bound = ref.STEP[dtype] * np.abs(want) + 1.01 * (K + 8) * ref.ACC * (A[expert[r]] @ np.abs(x64[r]))
        assert (np.abs(got[r] - want) <= bound + 1e-30).all(), r
    if E == 1:   # every row takes matrix 0
        valid = [r for r in range(R) if expert[r] == 0]
        again = moe.matvec_q4(x, q)["out"]
        assert torch.equal(again[valid], out[valid])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,N,K,E", [(3, 20000, 136, 1), (9, 40016, 136, 1), (64, 12944, 264, 64), (1, 48, 16520, 1),
                                     (4, 48, 8328, 1), (24, 32, 4232, 2)])
def test_matvec_many_strips_and_long_rows(R, N, K, E, dtype):
    """Work-groups of one, two and four waves, and several staged runs a wave."""
    say(f"matvec {dtype} R={R} N={N} K={K} E={E}")
    rng = np.random.default_rng(R + N)
    for group, kind, zero in ((64, "u4", True), (32, "e2m1", False)):
        codes, scale, z = ref.random_q4(rng, E, N, K, group, kind, zero)
        host = rng.standard_normal((R, K)).astype(np.float32)
        host = moe_inputs.to_bf16_bits(host) if dtype == "bf16" else host
        expert = rng.integers(0, E, R).astype(np.int32)
        q = moe.Q4Weights(torch.from_numpy(codes).cuda(), to_dev(scale, "bf16"),
                          None if z is None else torch.from_numpy(z).cuda(), (E, N, K), group, kind)
        out = moe.matvec_q4(to_dev(host, dtype), q, expert=torch.from_numpy(expert).cuda())["out"]
        torch.cuda.synchronize()
        got, x64 = bits_to_f64(to_host(out, dtype), dtype), bits_to_f64(host, dtype)
        s64 = moe_inputs.bits_to_f64(scale, "bf16")
        for e in np.unique(expert)[:3]:
            W, A = ref.q4_decode(codes[e:e + 1], s64[e:e + 1], None if z is None else z[e:e + 1], (1, N, K), group, kind)
            r = np.nonzero(expert == e)[0]
            want = x64[r] @ W[0].T
            bound = ref.STEP[dtype] * np.abs(want) + 1.01 * (K + 8) * ref.ACC * (np.abs(x64[r]) @ A[0].T)
            assert (np.abs(got[r] - want) <= bound + 1e-30).all(), e


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_infinite_inputs(dtype):
    """E2M1: an infinity times a weight is infinite, of its sign, and NaN where the weight is 0; U4: not finite.
    Other rows stay as they are."""
    w = torch.tensor([0.0, 1.0, -2.0, 6.0, -0.5, 3.0, 4.0, -1.5], device="cuda")[:, None].repeat(1, 40)[None].contiguous()
    x = torch.ones(3, 40, device="cuda", dtype=dtype)
    x[1, 37] = float("inf")
    got = moe.matvec_q4(x, moe.quantize_q4(w, group=32, kind="e2m1"))["out"].double()
    want = x.double() @ w[0].double().T
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.isnan(got[1, 0])
    assert torch.equal(torch.isinf(got), torch.isinf(want))
    assert torch.equal(got[1, 1:].sign(), want[1, 1:].sign())
    u4 = moe.quantize_q4(w, group=32, zero_points=False)
    a, b = moe.matvec_q4(x, u4)["out"], moe.matvec_q4(torch.ones_like(x), u4)["out"]
    assert not torch.isfinite(a[1]).any() and torch.equal(a[[0, 2]], b[[0, 2]])


def test_padding_is_not_looked_at():
    """NaN scales of rows past N and of groups that begin past K change nothing."""
    N, K, group = 20, 136, 32
    codes, scale, z = ref.random_q4(np.random.default_rng(5), 1, N, K, group, "u4", True)
    bad = scale.copy()
    bad[:, -1, :, N % 16:] = 0x7fc0
    bad[:, :, -(-K // group):] = 0x7fc0
    x = torch.randn(3, K, device="cuda").bfloat16()
    outs = []
    for s in (scale, bad):
        q = moe.Q4Weights(torch.from_numpy(codes).cuda(), to_dev(s, "bf16"), torch.from_numpy(z).cuda(), (1, N, K),
                          group, "u4")
        outs.append(moe.matvec_q4(x, q)["out"])
    assert torch.isfinite(outs[0]).all() and torch.equal(*outs)


def test_matvec_graph_and_streams():
    q = moe.quantize_q4(torch.randn(3, 200, 264, device="cuda"), group=32)
    x = torch.randn(9, 264, device="cuda")
    e = torch.tensor([0, 1, 2, 2, -1, 1, 0, 2, 1], dtype=torch.int32, device="cuda")
    want = moe.matvec_q4(x, q, expert=e)["out"].clone()
    assert (want[4] == 0).all()
    r = moe.matvec_q4(x, q, expert=e)
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        moe.matvec_q4(x, q, expert=e, out=r["out"], workspace=r["workspace"])
    for _ in range(3):
        r["out"].fill_(0)
        moe.matvec_q4(x * 2, q)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(r["out"], want)
    other = moe.matvec_q4(x, q, expert=e, stream=s)["out"]
    torch.cuda.synchronize()
    assert torch.equal(other, want)


def test_tensors_elsewhere_are_refused_by_name():
    q = moe.quantize_q4(torch.randn(1, 16, 64, device="cuda"), group=32)
    x = torch.randn(2, 64, device="cuda")
    for name, t in (("workspace", torch.empty(1 << 16, dtype=torch.uint8)), ("out", torch.empty(2, 16))):
        with pytest.raises(ValueError, match=name):
            moe.matvec_q4(x, q, **{name: t})
    with pytest.raises(ValueError, match="expert"):
        moe.matvec_q4(x, q, expert=torch.zeros(2, dtype=torch.int32))
