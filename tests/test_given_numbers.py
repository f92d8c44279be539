"""Numbers that a caller holds as tensors and changes in place between two calls: every call takes the value that it
finds. On the host, with stand-ins for the library and for a call's device and stream."""
import pytest

import routing_dispatch_expert_amd as moe
from tests.test_q4_weights import _Host

torch = pytest.importorskip("torch")


@pytest.fixture
def gates(monkeypatch):
    """What reaches the library's gate and its gradient, as (scale, groups, top_groups, group_best)."""
    seen = []

    class Lib:
        def moe_gate(self, logits, bias, gate, *a):
            g = gate.contents
            seen.append((g.scale, g.groups, g.top_groups, g.group_best))
            return 0

        def moe_gate_backward(self, logits, idx, dw, dscores, gate, *a):
            seen.append((gate.contents.scale,))
            return 0

    monkeypatch.setattr(moe, "lib", Lib)
    monkeypatch.setattr(moe, "_on", _Host)
    monkeypatch.setattr(moe, "_need", lambda *a: None)
    return seen


def test_gate_scale_changed_in_place(gates):
    logits, scale = torch.zeros(3, 8), torch.tensor(1.0)
    idx, w = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2)
    for want in (1.0, 2.5, 0.5):
        scale.fill_(want)
        moe.gate(logits, 2, scale=scale)
        moe.gate_backward(logits, idx, w, scale=scale)
        moe.moe_gate(logits, None, ("sigmoid", 1, 1, 1, 1, scale), 3, 8, 2, idx, w)
    assert [g[0] for g in gates] == [v for v in (1.0, 2.5, 0.5) for _ in range(3)]


def test_gate_groups_changed_in_place(gates):
    logits, groups, top, best = torch.zeros(3, 8), torch.tensor(2), torch.tensor(1), torch.tensor(1)
    for want in ((2, 1, 1), (4, 2, 2), (1, 1, 2)):
        for t, v in zip((groups, top, best), want):
            t.fill_(v)
        moe.gate(logits, 2, groups=groups, top_groups=top, group_best=best)
        assert gates[-1][1:] == want
