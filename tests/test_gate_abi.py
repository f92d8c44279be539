"""Refusals of the gate's entry points, on the host: every call fails its checks before any GPU work."""
import pytest

import routing_dispatch_expert_amd as moe

FAKE = 1 << 40   # never dereferenced
INVALID, UNSUPPORTED = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED


def rule(**kw):
    a = dict(score="sigmoid", groups=8, top_groups=4, group_best=2, renormalize=1, scale=2.5)
    a.update(kw)
    return tuple(a.values())


def call(**kw):
    a = dict(logits=FAKE, bias=None, gate=rule(), T=4, E=64, k=8, topk_idx=FAKE, topk_w=FAKE)
    a.update(kw)
    moe.moe_gate(**a)


def back(**kw):
    a = dict(logits=FAKE, topk_idx=FAKE, d_topk_w=FAKE, d_scores=None, gate=rule(), T=4, E=64, k=8, dlogits=FAKE * 2)
    a.update(kw)
    moe.moe_gate_backward(**a)


BOTH = [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(k=65), INVALID), (dict(gate=None), INVALID),
    (dict(logits=None), INVALID), (dict(topk_idx=None), INVALID), (dict(gate=rule(score=2)), INVALID),
    (dict(gate=rule(groups=0)), INVALID), (dict(gate=rule(groups=7)), INVALID), (dict(gate=rule(top_groups=0)), INVALID),
    (dict(gate=rule(top_groups=9)), INVALID), (dict(gate=rule(group_best=0)), INVALID), (dict(gate=rule(group_best=3)), INVALID),
    (dict(gate=rule(groups=64, group_best=2)), INVALID), (dict(gate=rule(groups=16, top_groups=1)), INVALID),
    (dict(gate=rule(scale=float("nan"))), INVALID), (dict(gate=rule(scale=float("inf"))), INVALID),
    (dict(E=8192, gate=rule(groups=1)), UNSUPPORTED), (dict(E=256, gate=rule(groups=128)), UNSUPPORTED),
    (dict(k=33), UNSUPPORTED), (dict(T=1 << 26), UNSUPPORTED), (dict(T=1 << 40), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", BOTH)
@pytest.mark.parametrize("fn", [call, back])
def test_refusals(fn, kw, status):
    with pytest.raises(moe.MoeError) as ei:
        fn(**kw)
    assert ei.value.status == status and moe.moe_last_error()


@pytest.mark.parametrize("fn,kw", [(call, dict(topk_w=None)), (back, dict(d_topk_w=None)), (back, dict(dlogits=None)),
                                   (back, dict(dlogits=FAKE + 64)), (back, dict(d_scores=FAKE * 2 + 64))])
def test_pointers(fn, kw):
    with pytest.raises(moe.MoeError) as ei:
        fn(**kw)
    assert ei.value.status == INVALID


def test_no_tokens():
    call(T=0, logits=None, topk_idx=None, topk_w=None)
    back(T=0, logits=None, topk_idx=None, d_topk_w=None, dlogits=None)


def test_python_refusals():
    torch = pytest.importorskip("torch")
    l = torch.zeros(2, 8)
    for bad in (lambda: moe.gate(l, 2), lambda: moe.gate(l[0], 2), lambda: moe.gate_backward(l, l[:, :2].int(), l[:, :2])):
        with pytest.raises(ValueError):   # not on a GPU, not two-dimensional
            bad()
