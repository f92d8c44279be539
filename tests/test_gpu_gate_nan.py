"""NaN and infinities among the gate's logits: what the formulas give, at every number of scores a lane holds."""
import numpy as np
import pytest

import routing_dispatch_expert_amd as moe
from tests import gate_reference as ref
from tests.gpu_util import U, gpu_available, say
from tests.test_gpu_gate import dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
SIZES = [8, 64, 65, 100, 256, 300, 700, 2000]   # 1, 2, 4, 8, 16 and 64 scores a lane


@pytest.fixture(autouse=True)
def _gpu():
    assert gpu_available(), "GPU tests need an MI355X; run them with -m gpu on a GPU host"
    moe.lib()


def rows(E):
    """Rows with: no NaN; one at the end of the order; all but two; nothing else; one of the other sign; +inf; +inf twice;
    one beside -inf; -inf alone."""
    l = np.random.default_rng(E).standard_normal((9, E)).astype(np.float32)
    l[1, E // 2] = np.nan
    l[2, 2:] = np.nan
    l[3] = np.nan
    l[4, E - 1] = -np.float32(np.nan)
    l[5, 3] = np.inf
    l[6, 1:3] = np.inf
    l[7] = -np.inf
    l[7, E - 2] = np.nan
    l[8] = -np.inf
    return l


def weights(l, idx, score, renormalize, scale):
    """The chosen ones' weights as the formulas have them, in 64 bits."""
    with np.errstate(all="ignore"):
        l = l.astype(np.float64)
        if score == "sigmoid":
            s = 1 / (1 + np.exp(-l))
        else:
            m = l.max(1, keepdims=True)   # NaN where there is one
            e = np.exp(l - np.where(np.isneginf(m), 0, m))
            total = e.sum(1, keepdims=True)
            s = e / np.where(total == 0, 1, total)
        z = np.take_along_axis(s, idx.astype(np.int64), 1)
        total = z.sum(1, keepdims=True)
        return scale * (z / np.where(total == 0, 1, total) if renormalize else z)


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", SIZES)
def test_weights(E, score, renormalize):
    say("gate with NaN", E, score, renormalize)
    l = rows(E)
    for k in (1, 4):
        for bias in (None, np.zeros(E, np.float32)):
            r = moe.gate(dev(l), k, score=score, bias=dev(bias), renormalize=renormalize, scale=1.5)
            idx, w = r["topk_idx"].cpu().numpy(), r["topk_w"].cpu().numpy()
            if bias is None:   # in the order of the logits, NaN last
                assert np.array_equal(idx, [ref._ranked(t)[:k] for t in l])
            want = weights(l, idx, score, renormalize, 1.5)
            assert np.array_equal(np.isnan(w), np.isnan(want)), (k, bias is None)
            ok = ~np.isnan(want)
            assert np.all(np.abs(w - want)[ok] <= U * (1 + 2.0 ** -20) * np.abs(want[ok]) + 2.0 ** -149)
            nan = np.array([1, 2, 3, 4, 5, 6, 7])
            assert np.isnan(w[nan]).all() if score == "softmax" else np.isnan(w[3]).all()
            assert not w[8].any()


def gradients(l, idx, dw, dsc, score, renormalize, scale):
    """Where the gradient is NaN, and the gradient of the rows without one, in 64 bits."""
    T, E = l.shape
    own = np.isnan(l)
    bad = ~(l < np.inf).all(1) if score == "softmax" else np.zeros(T, bool)   # every score of the row is NaN
    nan = np.zeros((T, E), bool)
    for t in range(T):
        if renormalize:   # the sum of the chosen ones' scores enters each of theirs
            nan[t, idx[t]] = bad[t] or own[t, idx[t]].any()
        elif score == "sigmoid":
            nan[t, idx[t]] = own[t, idx[t]]
        if dsc is not None or (score == "softmax" and not renormalize):
            nan[t] |= own[t] if score == "sigmoid" else bad[t]
    fine = ~(own.any(1) | bad)
    want, mag = np.zeros((T, E)), np.zeros((T, E))
    want[fine], mag[fine] = ref.gate_backward(l[fine], idx[fine], dw[fine], score, renormalize, scale, None if dsc is None else dsc[fine])
    return nan, want, mag, fine


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", SIZES)
def test_gradients(E, score, renormalize):
    say("gate backward with NaN", E, score, renormalize)
    rng = np.random.default_rng(E)
    l = rows(E)
    l[6, 1:3] = (-np.inf, 1.0)      # a row without NaN beside them
    for chosen in (False, True):    # whether the NaN is among the chosen
        order = [[e for e in ref._ranked(r) if chosen or np.isfinite(r[e])] for r in l]
        idx = np.array([(o[0], o[-1]) if len(o) > 1 else (0, 1) for o in order], np.int32)
        dw = rng.standard_normal(idx.shape).astype(np.float32)
        for dsc in (None, rng.standard_normal(l.shape).astype(np.float32)):
            got = moe.gate_backward(dev(l), dev(idx, np.int32), dev(dw), score=score, renormalize=renormalize, scale=1.5,
                                    d_scores=dev(dsc)).cpu().numpy()
            nan, want, mag, fine = gradients(l, idx, dw, dsc, score, renormalize, 1.5)
            assert np.array_equal(np.isnan(got), nan), (chosen, dsc is not None)
            steps = 2 * (E / 64 + 6 + 14)   # as in test_gpu_gate.py
            assert np.all(np.abs(got - want)[fine] <= U * steps * mag[fine] + 1e-38)
            assert not got[8].any()


@pytest.mark.parametrize("G,per", [(4, 8), (4, 16), (8, 32), (16, 40), (64, 3)])
def test_groups_of_nan_come_after_groups_of_masked_experts(G, per):
    """Group 1 has numbers, group 0 only NaN (or one number where two are added up), the others -inf (masked)."""
    E = G * per
    l = np.full((2, E), -np.inf, np.float32)
    l[:, per:2 * per] = np.random.default_rng(G).standard_normal(per)
    l[0, :per] = np.nan
    l[1, :per] = np.nan
    l[1, per // 2] = 3.0
    k = min(per + 2, 32)
    first = [per + i for i in ref._ranked(l[0, per:2 * per])]
    want = (first + list(range(2 * per, E)))[:k]
    r = moe.gate(dev(l), k, score="sigmoid", groups=G, top_groups=2)["topk_idx"].cpu().numpy()
    assert r[0].tolist() == want
    assert r[1, 0] == per // 2   # one number is enough for the largest
    bias = np.where(np.isneginf(l[0]), -np.inf, 0).astype(np.float32)
    for b in (None, bias):   # without a bias the scores are added up: those of -inf are 0
        r = moe.gate(dev(l), k, score="sigmoid", groups=G, top_groups=2, group_best=2, bias=dev(b))["topk_idx"].cpu().numpy()
        for row in r:
            assert row.tolist() == want
