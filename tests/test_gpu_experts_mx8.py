"""The experts with 8-bit rows and weights against 64 bits, on the GPU."""
import numpy as np
import pytest

import routing_dispatch_expert_amd as moe
from tests import mx8_reference as ref
from tests.gpu_util import U, gpu_available, say

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}   # half a step, relative
CUT = 2.0 ** -12   # what one instruction cuts off the sum of its products' magnitudes, at most


@pytest.fixture(autouse=True)
def _gpu():
    assert gpu_available(), "GPU tests need an MI355X; run them with -m gpu on a GPU host"
    moe.lib()


def slots(idx, E, C):
    out, count = np.full(idx.shape, -1, np.int32), np.zeros(E, np.int64)
    for at in np.ndindex(idx.shape):
        e = idx[at]
        if 0 <= e < E:
            if count[e] < C:
                out[at] = count[e]
            count[e] += 1
    return out, count


def matrix(gen, shape, ints, padding=127):
    """An Mx8 and its values: codes and scales of small whole numbers (ints), whose sums are exact, or of a Gaussian."""
    rng = gen
    K = shape[-1]
    groups = -(-K // 32)
    if ints:
        values = rng.integers(-1, 2, shape).astype(np.float64)
        byte = np.full((*shape[:-1], groups), 127) + (rng.integers(0, 2, (*shape[:-1], 1)))   # a row's scale 1 or 2
        codes = values
    else:
        codes = rng.standard_normal(shape) * 170
        codes = ref.values(np.clip(codes, -448, 448)) if K % 32 == 0 else np.clip(np.round(codes / 32) * 32, -448, 448)
        step = 2 * ref.half_step(codes)
        codes = np.clip(np.round(codes / step) * step, -448, 448)
        byte = 127 - 7 - round(np.log2(K) / 2) + rng.integers(-1, 2, (*shape[:-1], groups))
    packed = ref.pack_scale(byte, K)
    if groups % 4:
        packed[..., -1, :, groups % 4:] = padding     # bytes past the columns may be anything
    q = moe.Mx8(torch.from_numpy(codes).to(torch.float8_e4m3fn).cuda(), torch.from_numpy(packed).cuda())
    assert np.array_equal(q.codes.double().cpu().numpy(), codes)
    return q, codes * ref.two(ref.spread(byte, K))


def experts(x, Wg, Wu, Wd, idx, w, residual, C):
    """out - residual, the sum of its terms' magnitudes, what h's roundings may differ by in it, slots and counts, all
    in 64 bits. h = silu(g) u of exact g and u is off by 2^-21 of itself (an exponential, a sum, a quotient and a product in
    fp32: 2^-24 each and one more for the exponential's argument): where that reaches over the middle between two
    numbers of the 8-bit grid (whole g past 17 have silu(g) = g in fp32, and h lies on such middles), either is right."""
    E = Wg.shape[0]
    slot, count = slots(idx, E, C)
    part = np.zeros(residual.shape)
    size = np.zeros(residual.shape)
    slack = np.zeros(residual.shape)
    for e in range(E):
        t, j = np.nonzero((idx == e) & (slot >= 0))
        if not len(t):
            continue
        g, u = x[t] @ Wg[e].T, x[t] @ Wu[e].T
        h = g / (1 + np.exp(-g)) * u
        either = np.abs(ref.values(h * (1 + 2.0 ** -21)) - ref.values(h * (1 - 2.0 ** -21)))
        h = ref.values(h)
        np.add.at(slack, t, np.abs(w[t, j][:, None]) * (either @ np.abs(Wd[e]).T))
        np.add.at(part, t, w[t, j][:, None] * (h @ Wd[e].T))
        np.add.at(size, t, np.abs(w[t, j][:, None]) * (np.abs(h) @ np.abs(Wd[e]).T))
    return part, size, slack, slot, count


def route(rng, T, E, k):
    return np.argsort(rng.random((T, E)), 1)[:, :k].astype(np.int32)


def run_case(T, d, f, E, k, cf, dtype="bf16", ints=True, idx=None, padding=127, seed=0):
    say("experts", T, d, f, E, k, cf, dtype, "whole numbers" if ints else "Gaussian")
    rng = np.random.default_rng(seed + T + d + f + E)
    idx = route(rng, T, E, k) if idx is None else idx
    w = rng.random((T, k)).astype(np.float32) - 0.2
    (xq, x), (gq, Wg), (uq, Wu), (dq, Wd) = (matrix(rng, s, ints, padding) for s in ((T, d), (E, f, d), (E, f, d), (E, d, f)))
    residual = torch.from_numpy(rng.standard_normal((T, d))).to(DT[dtype]).cuda()
    r = moe.experts_mx8(xq, torch.from_numpy(idx).cuda(), torch.from_numpy(w).cuda(), gq, uq, dq, residual, cf)
    C = moe.moe_capacity(T, E, k, cf)
    part, size, slack, slot, count = experts(x, Wg, Wu, Wd, idx, w.astype(np.float64), residual.double().cpu().numpy(), C)
    assert np.array_equal(r["slot"].cpu().numpy(), slot)
    assert np.array_equal(r["routed_count"].cpu().numpy(), count)
    assert np.array_equal(r["kept_count"].cpu().numpy(), np.minimum(count, C))
    out, base = r["out"].double().cpu().numpy(), residual.double().cpu().numpy()
    left = (slot < 0).all(1)
    same = np.array_equal(out[left], base[left])   # nothing kept: as it was
    assert same
    if ints:
        # g and u are exact, h as above; y is cut in each instruction, rounded, and summed over k
        off = (CUT + HALF[dtype] + U * (k + f / 64 + 8)) * (size + slack) + slack
        bad = np.abs(out - (base + part)) > off + HALF[dtype] * (np.abs(base + part) + off)
        assert not bad.any(), f"{bad.sum()} of {bad.size}, first {np.argwhere(bad)[:5].tolist()}"
    else:
        # g and u are off by 2^-16 of their size (sums of cut products: 1.3e-5 over 4096 columns), so that one h in some
        # thousand rounds to its other neighbour, 2^-3 of it away: 2^-8 of the sum's norm; y is rounded once more
        off = np.linalg.norm(out - base - part, axis=1)
        most = (2.0 ** -7 + 2 * HALF[dtype]) * np.linalg.norm(part, axis=1) + HALF[dtype] * np.linalg.norm(out, axis=1)
        assert not (off > most).any(), f"rows {np.flatnonzero(off > most)[:8]}, {(off / most).max()} times"
    return r


SIZES = [(1, 16, 16, 1, 1, 1.0), (1, 128, 64, 4, 2, 2.0), (3, 144, 48, 4, 2, 2.0), (5, 272, 80, 3, 3, 1.0), (17, 128, 32, 1, 1, 1.0),
         (33, 256, 96, 2, 1, 2.0), (70, 400, 144, 4, 2, 1.0), (64, 512, 160, 12, 3, 0.5), (130, 640, 176, 2, 2, 1.0),
         (1, 2048, 1408, 8, 6, 2.0), (300, 256, 256, 4, 2, 0.7), (520, 128, 384, 2, 1, 2.0), (700, 384, 272, 3, 2, 1.25)]


@pytest.mark.parametrize("ints", [True, False], ids=["whole", "gauss"])
@pytest.mark.parametrize("T,d,f,E,k,cf", SIZES)
def test_experts(T, d, f, E, k, cf, ints):
    run_case(T, d, f, E, k, cf, ints=ints)


# rows an expert on both sides of the rules for strips, tiles of 128 rows and of 256; one to seven 128-column steps, whole and not
STEPS = [(50, 128, 128, 2, 2, 1.0), (100, 768, 384, 4, 2, 2.0), (90, 640, 896, 4, 2, 2.0), (60, 400, 272, 3, 1, 3.0),
         (400, 512, 896, 2, 1, 2.0), (300, 128, 768, 2, 1, 2.0), (384, 144, 656, 4, 1, 4.0), (388, 656, 144, 4, 1, 4.0),
         (80, 256, 528, 4, 1, 4.0), (84, 528, 256, 4, 1, 4.0), (16, 272, 4112, 1, 1, 1.0), (25, 2064, 48, 1, 1, 1.0)]


@pytest.mark.parametrize("ints", [True, False], ids=["whole", "gauss"])
@pytest.mark.parametrize("T,d,f,E,k,cf", STEPS)
def test_steps_and_rules(T, d, f, E, k, cf, ints):
    run_case(T, d, f, E, k, cf, ints=ints)


# down's tiles split over K: 48 steps (the fewest) to 65, whole and not, in two to four parts; rows that end inside a tile;
# live tiles that are no multiple of eight
DEEP = [(300, 272, 6160, 2, 1, 2.0, "bf16"), (220, 144, 6144, 1, 1, 1.0, "f32"), (700, 640, 8208, 4, 2, 0.7, "bf16"),
        (260, 2064, 6400, 1, 1, 1.0, "f32"), (129, 528, 8192, 2, 2, 1.0, "bf16"),
        # the same with tiles of 128 rows: 25 to 96 rows an expert
        (50, 272, 6160, 2, 1, 2.0, "bf16"), (96, 144, 6144, 1, 1, 1.0, "f32"), (65, 640, 8208, 4, 2, 0.7, "bf16"),
        (70, 2064, 6400, 2, 1, 2.0, "f32")]


@pytest.mark.parametrize("ints", [True, False], ids=["whole", "gauss"])
@pytest.mark.parametrize("T,d,f,E,k,cf,dtype", DEEP)
def test_down_split_over_its_columns(T, d, f, E, k, cf, dtype, ints):
    run_case(T, d, f, E, k, cf, dtype, ints=ints)


@pytest.mark.parametrize("T", [4400, 4230])
def test_whole_rounds_and_a_split_rest(T):
    """288 and 272 tiles of down: 36 and 34 an XCD, of which 32 are whole. A sample of tokens against 64 bits, all of them
    twice the same, and in a graph whose replays find other numbers in the workspace."""
    d, f = 4096, 6144
    rng = np.random.default_rng(T)
    (xq, x), (gq, Wg), (uq, Wu), (dq, Wd) = (matrix(rng, s, True) for s in ((T, d), (1, f, d), (1, f, d), (1, d, f)))
    idx = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    w = torch.full((T, 1), 0.5, device="cuda")
    residual = torch.zeros((T, d), dtype=torch.bfloat16, device="cuda")
    run = lambda: moe.experts_mx8(xq, idx, w, gq, uq, dq, residual, 1.0)["out"]
    say("experts, split rest", T, d, f)
    out = run()
    pick = np.unique(np.concatenate([rng.integers(0, T, 60), [0, 1, 255, 256, T - 257, T - 256, T - 2, T - 1]]))
    g, u = x[pick] @ Wg[0].T, x[pick] @ Wu[0].T
    h = g / (1 + np.exp(-g)) * u
    either = np.abs(ref.values(h * (1 + 2.0 ** -21)) - ref.values(h * (1 - 2.0 ** -21)))
    h = ref.values(h)
    part, size, slack = (0.5 * v @ np.abs(Wd[0]).T if v is not h else 0.5 * h @ Wd[0].T for v in (h, np.abs(h), either))
    off = (CUT + HALF["bf16"] + U * (1 + f / 64 + 8)) * (size + slack) + slack   # as run_case()
    got = out.double().cpu().numpy()[pick]
    bad = np.abs(got - part) > off + HALF["bf16"] * (np.abs(part) + off)
    assert not bad.any(), f"{bad.sum()} of {bad.size}, first {np.argwhere(bad)[:5].tolist()}"
    assert torch.equal(out, run())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = run()
    for _ in range(3):
        again.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, again)
        run()


@pytest.mark.parametrize("T,E", [(100, 64), (33, 64), (300, 4), (700, 8)])
def test_one_expert_with_many_rows_among_experts_with_few(T, E):
    """Strips take such an expert 32 rows at a time, tiles by more of them."""
    rng = np.random.default_rng(T)
    idx = np.full((T, 1), E // 2, np.int32)
    few = rng.permutation(T)[:E // 2]
    idx[few, 0] = np.arange(E // 2)
    run_case(T, 144, 80, E, 1, float(E), idx=idx)
    run_case(T, 144, 80, E, 1, float(E), idx=idx, ints=False)


@pytest.mark.parametrize("ints", [True, False], ids=["whole", "gauss"])
@pytest.mark.parametrize("T,d,f,E,k,cf", [(2, 144, 80, 4, 2, 2.0), (40, 256, 96, 2, 2, 1.0), (400, 272, 176, 2, 1, 2.0)])
def test_experts_fp32(T, d, f, E, k, cf, ints):
    run_case(T, d, f, E, k, cf, dtype="f32", ints=ints)


@pytest.mark.parametrize("T", [2, 40, 300])
def test_bytes_past_the_columns_may_be_nan(T):
    run_case(T, 144, 80, 2, 1, 2.0, padding=255)
    run_case(T, 48, 48, 2, 1, 2.0, padding=255, ints=False)


@pytest.mark.parametrize("T,hot", [(5, 3), (100, 0), (600, 2)])
def test_every_copy_to_one_expert(T, hot):
    idx = np.full((T, 1), hot, np.int32)
    run_case(T, 128, 64, 4, 1, 4.0, idx=idx)
    run_case(T, 128, 64, 4, 1, 1.0, idx=idx)       # three quarters dropped


@pytest.mark.parametrize("T", [6, 80, 500])
def test_outside_and_repeated_indices(T):
    rng = np.random.default_rng(T)
    idx = route(rng, T, 5, 3)
    idx[0] = (-1, 5, 1 << 30)                       # no expert at all
    idx[1] = (2, 2, 2)
    idx[2::3, 1] = -(1 << 31)
    run_case(T, 160, 96, 5, 3, 5 / 3, idx=idx)
    run_case(T, 160, 96, 5, 3, 0.6, idx=idx)


@pytest.mark.parametrize("T,E,k", [(9, 4096, 2), (40, 1000, 32), (300, 300, 8), (33, 1, 1), (2000, 64, 6)])
def test_lists_of_many_experts(T, E, k):
    run_case(T, 16, 16, E, k, E / k if E <= 1000 else 600.0)


def test_nan_stays_with_its_expert_and_token():
    """A NaN in one expert's weights or one token's rows reaches no other."""
    rng = np.random.default_rng(3)
    T, d, f, E = 40, 256, 96, 3
    idx = np.arange(T, dtype=np.int32)[:, None] % E
    mats = [matrix(rng, s, True)[0] for s in ((T, d), (E, f, d), (E, f, d), (E, d, f))]
    residual, w = torch.zeros(T, d, device="cuda"), torch.ones(T, 1, device="cuda")
    call = lambda: moe.experts_mx8(mats[0], torch.from_numpy(idx).cuda(), w, *mats[1:], residual, 3.0)["out"]  # noqa: E731
    want = call()
    mats[2].scale[1, 0, 5, 2] = 255
    got = call()
    ok = torch.from_numpy(idx[:, 0] != 1).cuda()
    assert torch.equal(got[ok], want[ok]) and got[~ok].isnan().all()
    mats[2].scale[1, 0, 5, 2] = 127
    mats[0].codes.view(torch.uint8)[6, 100] = 127
    got = call()
    ok = torch.arange(T, device="cuda") != 6
    assert torch.equal(got[ok & (torch.arange(T, device="cuda") % 3 != 1)], want[ok & (torch.arange(T, device="cuda") % 3 != 1)])
    assert got[6].isnan().all()


def test_lent_outputs_and_rows_behind_the_batch():
    rng = np.random.default_rng(5)
    r = run_case(40, 128, 64, 4, 2, 2.0)
    (x, _), (g, _), (u, _), (dn, _) = (matrix(rng, s, True) for s in ((40, 128), (4, 64, 128), (4, 64, 128), (4, 128, 64)))
    idx, w = torch.from_numpy(route(rng, 40, 4, 2)).cuda(), torch.rand(40, 2, device="cuda")
    res = torch.randn(40, 128, device="cuda").bfloat16()
    a = moe.experts_mx8(x, idx, w, g, u, dn, res, 2.0)
    b = moe.experts_mx8(x, idx, w, g, u, dn, res, 2.0, out=r)
    assert b is r and torch.equal(a["out"], b["out"]) and torch.equal(a["slot"], b["slot"])
    for kw in (dict(cf=1.0), dict(residual=res.float())):
        with pytest.raises(ValueError):
            moe.experts_mx8(x, idx, w, g, u, dn, **{**dict(residual=res, cf=2.0, out=r), **kw})
    # in place, with guarded rows behind
    n = moe.moe_experts_mx8_workspace_size(40, 128, 64, 4, 2, 2.0, "bf16")
    ws = torch.full((n + 4096,), 77, dtype=torch.uint8, device="cuda")
    behind = torch.full((48, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    behind[:40] = res
    moe.moe_experts_mx8(x, behind, idx, w, g, u, dn, 40, 128, 64, 4, 2, 2.0, "bf16", behind, None, ws, n, torch.cuda.current_stream())
    assert torch.equal(behind[:40], a["out"]) and (behind[40:] == 5).all() and (ws[n:] == 77).all()
    e = moe.experts_mx8(moe.quantize_mx8(torch.zeros(0, 128, device="cuda")), idx[:0], w[:0], g, u, dn, res[:0], 2.0)
    assert e["out"].shape == (0, 128) and not e["kept_count"].any()


def test_the_same_call_gives_the_same_bits():
    rng = np.random.default_rng(9)
    for T in (7, 500):
        (x, _), (g, _), (u, _), (dn, _) = (matrix(rng, s, False) for s in ((T, 512), (6, 256, 512), (6, 256, 512), (6, 512, 256)))
        idx, w = torch.from_numpy(route(rng, T, 6, 2)).cuda(), torch.rand(T, 2, device="cuda")
        res = torch.randn(T, 512, device="cuda")
        want = moe.experts_mx8(x, idx, w, g, u, dn, res, 3.0)["out"]
        for _ in range(5):
            assert torch.equal(moe.experts_mx8(x, idx, w, g, u, dn, res, 3.0)["out"], want)
