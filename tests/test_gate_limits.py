"""The largest sizes of the gate's entry points as moe.h states them, on the host: the last that passes the checks (and
is then refused for its missing tensors) and the first that does not."""
import pytest

import routing_dispatch_expert_amd as moe
from tests.test_gate_abi import INVALID, UNSUPPORTED, back, call, rule

NONE = dict(gate=rule(groups=1))


@pytest.mark.parametrize("inside,outside", [(dict(T=(1 << 26) - 5), dict(T=(1 << 26) - 4)), (dict(E=4096), dict(E=4104)),
                                            (dict(E=64, k=32), dict(E=64, k=33)),
                                            (dict(T=(1 << 26) - 5, E=64, k=31), dict(T=1 << 26, E=64, k=32)),
                                            (dict(E=640, gate=rule(groups=64)), dict(E=650, gate=rule(groups=65)))], ids=str)
@pytest.mark.parametrize("fn", [call, back])
def test_limits(fn, inside, outside):
    for kw, status in ((inside, INVALID), (outside, UNSUPPORTED)):
        with pytest.raises(moe.MoeError) as ei:
            fn(**{**NONE, **kw, "logits": None})
        assert ei.value.status == status
