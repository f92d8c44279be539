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


class _Calls:
    """Runs the Python side of a call on host tensors and keeps what would have reached the library."""

    def __init__(self, monkeypatch):
        self.seen = []
        for name in ("_on", "_On"):
            monkeypatch.setattr(moe, name, _Host)
        for name in ("_need", "_require"):
            monkeypatch.setattr(moe, name, lambda *a: None)
        for name in ("moe_layer_forward_routed", "moe_layer_backward_routed", "moe_layer_forward_few", "moe_experts_mx8", "moe_rmsnorm",
                     "moe_router", "moe_gate"):
            monkeypatch.setattr(moe, name, lambda *a: self.seen.append(a))
        z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t)  # noqa: E731
        q = lambda *s: moe.Mx8(z(*s, t=torch.float8_e4m3fn), z(*s[:-2], 1, s[-2], 4, t=torch.uint8))  # noqa: E731
        self.x, self.Wr, self.idx, self.w = z(16, 64), z(8, 64), z(16, 2, t=torch.int32), z(16, 2, t=torch.float32)
        self.W = [z(8, 32, 64), z(8, 32, 64), z(8, 64, 32)]
        self.q, self.x8 = [q(8, 32, 64), q(8, 32, 64), q(8, 64, 32)], q(16, 64)

    def routed(self, k, cf, P, out):
        return moe.forward_routed(self.x, self.idx, self.w, *self.W, cf=cf, P=P, keep_activations=True, out=out)

    def routed_backward(self, k, cf, P, out):
        return moe.backward_routed(self.x, self.idx, self.w, *self.W, self.x, cf=cf, P=P, out=out)

    def few(self, k, cf, P, out):
        return moe.forward_few(self.x, self.Wr, *self.W, k=k, cf=cf, P=P, out=out)

    def experts(self, k, cf, P, out):
        return moe.experts_mx8(self.x8, self.idx, self.w, *self.q, residual=self.x, cf=cf, out=out)

    def block(self, k, cf, P, out):
        return moe.forward_mx8(self.x, self.Wr[0], self.Wr, *self.q, k=k, cf=cf, out=out)

    def gate(self, k, cf, P, out):
        return moe.gate(self.Wr.float(), k, out=out)


@pytest.mark.parametrize("name,numbers", [("routed", ("cf", "P")), ("routed_backward", ("cf", "P")), ("few", ("k", "cf", "P")),
                                          ("experts", ("cf",)), ("block", ("k", "cf")), ("gate", ("k",))])
def test_a_lent_result_is_of_the_numbers_it_was_made_with(name, numbers, monkeypatch):
    """Its tensors are as large as k, cf and P asked for then: after a change in place it is refused as any other of
    another size is, and the same numbers, held as tensors or not, take it."""
    calls = _Calls(monkeypatch)
    for changed in numbers:
        n = dict(k=torch.tensor(2), cf=torch.tensor(1.0), P=torch.tensor(2))
        out = getattr(calls, name)(**n, out=None)
        assert getattr(calls, name)(**n, out=out) is out
        assert getattr(calls, name)(k=2, cf=1.0, P=2, out=out) is out
        n[changed].mul_(2)
        done = len(calls.seen)
        with pytest.raises(ValueError, match="out"):
            getattr(calls, name)(**n, out=out)
        assert len(calls.seen) == done   # nothing reached the library


def test_a_kept_state_is_of_the_numbers_it_was_made_with(monkeypatch):
    calls = _Calls(monkeypatch)
    for changed in ("cf", "P"):
        n = dict(cf=torch.tensor(1.0), P=torch.tensor(2))
        saved = calls.routed(2, n["cf"], n["P"], None)
        call = lambda: moe.backward_routed(calls.x, calls.idx, calls.w, *calls.W, calls.x, **n, saved=saved)  # noqa: E731
        call()
        n[changed].mul_(2)
        with pytest.raises(ValueError, match="saved"):
            call()
