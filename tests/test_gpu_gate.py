"""The gate (scores, balance bias, groups, top-k, weights) and its gradient
against 64 bits, on the GPU."""
import numpy as np
import pytest

import routing_dispatch_expert_amd as moe
from tests import gate_reference as ref
from tests.gpu_util import U, gpu_available, say

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    assert gpu_available(), "GPU tests need an MI355X; run them with -m gpu on a GPU host"
    moe.lib()


def dev(a, dtype=np.float32):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype)).cuda()


def check(l, k, bias=None, **kw):
    r = moe.gate(dev(l), k, bias=dev(bias), **kw)
    idx, w = ref.gate(l, k, bias=bias, **kw)
    assert np.array_equal(r["topk_idx"].cpu().numpy(), idx)
    # 64-bit evaluation, rounded once (half a step of fp32 is 2^-24) and below 2^-126 to a multiple of 2^-149
    assert np.all(np.abs(r["topk_w"].cpu().numpy() - w) <= U * (1 + 2.0 ** -20) * np.abs(w) + 2.0 ** -149)
    return r


SHAPES = [(1, 1, 1), (1, 4, 2), (3, 60, 6), (5, 64, 8), (129, 72, 1), (65, 128, 16), (1000, 256, 8), (2, 300, 32), (9, 512, 7),
          (4, 1000, 10), (3, 2048, 8), (2, 4096, 32)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_gate(T, E, k, score):
    rng = np.random.default_rng(T + E + k)
    l = (1.5 * rng.standard_normal((T, E))).astype(np.float32)
    b = (0.05 * rng.standard_normal(E)).astype(np.float32)
    for bias in (None, b):
        for renormalize, scale in ((True, 1.0), (False, 2.5), (True, 2.5)):
            say("gate", T, E, k, score, bias is not None, renormalize)
            check(l, k, bias, score=score, renormalize=renormalize, scale=scale)


GROUPS = [(7, 8, 2, 4, 2), (33, 256, 8, 8, 4), (5, 60, 6, 5, 2), (3, 72, 4, 3, 1), (4, 128, 2, 64, 3), (2, 4096, 16, 8, 3),
          (6, 192, 6, 6, 6), (3, 1000, 5, 20, 2), (2, 126, 3, 63, 2), (3, 1088, 2, 17, 2)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,G,M", GROUPS)
def test_groups(T, E, k, G, M, score):
    rng = np.random.default_rng(E + G)
    l = (1.5 * rng.standard_normal((T, E))).astype(np.float32)
    b = (0.05 * rng.standard_normal(E)).astype(np.float32)
    for bias in (None, b):
        for best in (1, 2) if E // G > 1 else (1,):
            say("groups", T, E, k, G, M, score, bias is not None, best)
            check(l, k, bias, score=score, groups=G, top_groups=M, group_best=best, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_go_to_the_lower_index(score):
    rng = np.random.default_rng(5)
    l = rng.integers(-2, 3, (64, 96)).astype(np.float32)
    l[l == 0] *= rng.choice((-1.0, 1.0), np.count_nonzero(l == 0))   # +0 and -0 are equal
    for kw in ({}, dict(bias=np.zeros(96, np.float32)), dict(groups=8, top_groups=3),
               dict(groups=8, top_groups=3, group_best=2, bias=np.zeros(96, np.float32))):
        check(l, 8, score=score, **kw)
    check(np.zeros((3, 256), np.float32), 8, score=score, groups=8, top_groups=4, group_best=2)


def test_scores_that_fp32_cannot_tell_apart():
    """Scores some 2^-30 apart, through the bias: equal in fp32, in order in 64 bits."""
    l = np.zeros((1, 64), np.float32)
    bias = (np.arange(64) * 2.0 ** -34).astype(np.float32)
    r = check(l, 8, bias, score="sigmoid")
    assert r["topk_idx"].cpu().tolist() == [list(range(63, 55, -1))]


@pytest.mark.parametrize("G,E", [(2, 64), (2, 8), (2, 130), (3, 48), (4, 64), (5, 80), (8, 64), (9, 72), (16, 64), (32, 64)])
def test_the_two_largest_of_a_group_wherever_they_lie(G, E):
    """One token per pair of places: group 1 wins by the sum of exactly these two, group 0 has the one largest."""
    per = E // G
    pairs = [(a, c) for a in range(per) for c in range(a)]
    l = np.full((len(pairs), E), -2.0, np.float32)
    l[:, 0] = 2.0                             # sigmoid: 0.881 + 0.119 in group 0
    for t, (a, c) in enumerate(pairs):
        l[t, per + a], l[t, per + c] = 1.0, 0.5   # 0.731 + 0.622 in group 1
    r = check(l, 2, score="sigmoid", groups=G, top_groups=1, group_best=2)
    assert np.array_equal(r["topk_idx"].cpu().numpy(), [[per + a, per + c] for a, c in pairs])
    r = check(l, 2, score="sigmoid", groups=G, top_groups=1)   # by the largest alone
    assert np.all(r["topk_idx"].cpu().numpy()[:, 0] == 0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("step", [2.0 ** -e for e in (27, 24, 22, 21, 20, 19, 18, 17, 16, 14)])
def test_scores_that_lie_close(step, score):
    """Values in random order, steps apart that fp32 cannot, can hardly and can tell: the order is that of 64 bits."""
    rng = np.random.default_rng(8)
    l = (0.5 * rng.standard_normal((40, 256))).astype(np.float32)
    s = ref.scores(l[:1], score)
    for level in (0.5, 40.0):
        bias = (level + step * rng.permutation(256) - s[0]).astype(np.float32)   # the first row's values: level + steps
        for kw in ({}, dict(groups=8, top_groups=4, group_best=2), dict(groups=16, top_groups=3)):
            check(l, 8, bias, score=score, scale=1.5, **kw)
    near = (np.round(l / step) * step).astype(np.float32)
    check(near, 8, score=score)
    check(near, 8, score=score, groups=8, top_groups=2, group_best=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_masked_rows_and_large_logits(score, renormalize):
    rng = np.random.default_rng(6)
    l = rng.standard_normal((8, 100)).astype(np.float32)
    l[0] = -np.inf                               # nothing left
    l[1, 3:] = -np.inf                           # fewer left than are chosen
    l[2, ::2] = -np.inf
    l[3] = np.finfo(np.float32).min              # the type's lowest value
    l[4] *= 300
    l[5] = -200 + l[5]
    l[6, :50] = np.finfo(np.float32).min
    for bias in (None, np.zeros(100, np.float32)):
        for kw in ({}, dict(groups=10, top_groups=2, group_best=2)):
            check(l, 8, bias, score=score, renormalize=renormalize, **kw)
    assert not moe.gate(dev(l), 8, score=score, renormalize=renormalize)["topk_w"][0].any()


@pytest.mark.parametrize("kw", [{}, dict(groups=8, top_groups=2, group_best=2), dict(groups=8, top_groups=2)], ids=str)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_nan_and_infinities_leave_distinct_experts(score, kw):
    rng = np.random.default_rng(7)
    l = rng.standard_normal((6, 64)).astype(np.float32)
    l[0] = np.nan
    l[1, ::3] = np.nan
    l[2, 5] = np.inf
    l[3] = np.inf
    l[4, :] = np.where(rng.random(64) < 0.5, np.inf, -np.inf)
    l[5, 60:] = np.nan
    for bias in (None, np.full(64, np.nan, np.float32), np.zeros(64, np.float32)):
        i = moe.gate(dev(l), 8, score=score, bias=dev(bias), **kw)["topk_idx"].cpu().numpy()
        assert ((i >= 0) & (i < 64)).all() and all(len(set(r)) == 8 for r in i)


def _backward_case(T, E, k, seed):
    rng = np.random.default_rng(seed)
    l = (1.5 * rng.standard_normal((T, E))).astype(np.float32)
    idx = np.argsort(rng.random((T, E)), 1)[:, :k].astype(np.int32)
    return l, idx, rng.standard_normal((T, k)).astype(np.float32), (0.1 * rng.standard_normal((T, E))).astype(np.float32)


def check_backward(l, idx, dw, dsc, **kw):
    got = moe.gate_backward(dev(l), dev(idx, np.int32), dev(dw), d_scores=dev(dsc), **kw).cpu().numpy()
    want, mag = ref.gate_backward(l, idx, dw, d_scores=dsc, **kw)
    # the chosen ones' terms are rounded from 64 bits; a dense term has the rounding of expf (2 steps), of the sums over
    # E / 64 values a lane and 6 levels of lanes, and of some ten products, each of the magnitudes that enter it; twice for the lot
    steps = 2 * (l.shape[1] / 64 + 6 + 14)
    assert np.all(np.abs(got - want) <= U * steps * mag + 1e-38)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 4, 1), (3, 64, 6), (130, 100, 8), (7, 256, 8), (5, 333, 3), (3, 700, 12), (2, 4096, 32)])
def test_backward(T, E, k, score, renormalize):
    l, idx, dw, dsc = _backward_case(T, E, k, T + E)
    for d in (None, dsc):
        say("gate backward", T, E, k, score, renormalize, d is not None)
        check_backward(l, idx, dw, d, score=score, renormalize=renormalize, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_backward_against_differences(score, renormalize):
    l, idx, dw, dsc = _backward_case(4, 40, 5, 3)
    got = moe.gate_backward(dev(l), dev(idx, np.int32), dev(dw), score=score, renormalize=renormalize, scale=1.5,
                            d_scores=dev(dsc)).cpu().numpy()

    def loss(l):
        s = ref.scores(l, score)
        w = np.take_along_axis(s, idx, 1)
        w = w / w.sum(1, keepdims=True) if renormalize else w
        return (1.5 * w * dw).sum() + (s * dsc).sum()

    step = 1e-5   # a central difference's own error: step^2 times a third derivative of order 1, and 2^-53 / step
    for t in range(4):
        for e in range(40):
            a, b = l.astype(np.float64), l.astype(np.float64)
            a[t, e] += step
            b[t, e] -= step
            assert abs((loss(a) - loss(b)) / (2 * step) - got[t, e]) < 1e-6


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_backward_of_repeated_and_outside_indices(score, renormalize):
    l, idx, dw, dsc = _backward_case(6, 70, 4, 9)
    idx[0, 1] = idx[0, 0]
    idx[1, :] = 69
    idx[2, 2], idx[3, 0], idx[4] = -1, 70, (-5, 1 << 30, -(1 << 31), 70)
    for d in (None, dsc):
        check_backward(l, idx, dw, d, score=score, renormalize=renormalize, scale=1.0)


def test_backward_of_masked_rows():
    l, idx, dw, dsc = _backward_case(3, 64, 4, 11)
    l[0] = -np.inf
    l[1, 10:] = -np.inf
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            for d in (None, dsc):
                got = moe.gate_backward(dev(l), dev(idx, np.int32), dev(dw), score=score, renormalize=renormalize, d_scores=dev(d))
                assert not got[0].any() and torch.isfinite(got).all() and not got[1, 10:].any()


def test_lent_outputs_and_empty_batches():
    l = dev(np.random.default_rng(1).standard_normal((5, 32)))
    r = moe.gate(l, 4)
    at = r["topk_idx"].data_ptr()
    want = r["topk_idx"].clone()
    r["topk_idx"] = None
    again = moe.gate(l, 4, out=r)
    assert again["topk_idx"].data_ptr() == at and torch.equal(again["topk_idx"], want)
    with pytest.raises(ValueError):
        moe.gate(l, 5, out=r)
    e = moe.gate(l[:0], 4, groups=4, top_groups=2)
    assert e["topk_idx"].shape == (0, 4)
    assert moe.gate_backward(l[:0], e["topk_idx"], e["topk_w"]).shape == (0, 32)
