"""silu in the 8-bit experts over the whole range of fp32: g and u one number each, h seen through one column of W_down."""
import numpy as np
import pytest

import routing_dispatch_expert_amd as moe
from tests import mx8_reference as ref
from tests.gpu_util import gpu_available, say

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    assert gpu_available(), "GPU tests need an MI355X; run them with -m gpu on a GPU host"
    moe.lib()


# g and u as code times 2^e
HUGE = [((c, 127), (1.5, -e)) for c in (1.0, 1.25, 1.5, 1.75, -1.0, -1.75) for e in (127, 120, 60)]
LARGE = [((c, e), (-1.25, 30)) for c in (1.125, -1.125) for e in (7, 8, 10, 30, 60, 90)]
SMALL = [((c, 0), (u, e)) for c in (-80, -88, -96, -104, -120, -144, -208, 88, 96, 104, 144) for u, e in ((1.0, 0), (1.75, 100), (-1.0, -100))]
CASES = HUGE + LARGE + SMALL + [((c, -3), (1.0, 0)) for c in (-448, -100, -9, -1, 0, 1, 9, 100, 448)]


@pytest.mark.parametrize("at", range(0, len(CASES), 12))
def test_in_strips(at):
    check(CASES[at:at + 12])


@pytest.mark.parametrize("copies", [1, 3])   # tiles of 128 rows and of 256
def test_in_tiles(copies):
    check(CASES * copies)


def check(cases):
    say("silu", len(cases))
    T, d, f = len(cases), 128, 32
    codes, byte = np.zeros((T, d)), np.full((T, 4), 127)
    for t, (g, u) in enumerate(cases):
        (codes[t, 0], e), (codes[t, 32], byte_u) = g, u
        byte[t, :2] = 127 + e, 127 + byte_u
    mats = []
    for at, shape in ((0, (1, f, d)), (32, (1, f, d)), (0, (1, d, f))):
        w = np.zeros(shape)
        w[:, :, at] = 1
        mats.append(moe.Mx8(torch.from_numpy(w).to(torch.float8_e4m3fn).cuda(), torch.full((1, 1, shape[1], 4), 127, dtype=torch.uint8).cuda()))
    x8 = torch.from_numpy(codes).to(torch.float8_e4m3fn).cuda()
    assert np.array_equal(x8.double().cpu().numpy(), np.array([[ref.decode(b) for b in r] for r in x8.view(torch.uint8).cpu().numpy()]))
    x = moe.Mx8(x8, torch.from_numpy(ref.pack_scale(byte, d)).cuda())
    one, zero = torch.ones(T, 1, device="cuda"), torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    out = moe.experts_mx8(x, zero, one, *mats, torch.zeros(T, d, device="cuda"), 1.0)["out"].double().cpu().numpy()
    c = x8.double().cpu().numpy()
    g, u = (c[:, 32 * i] * 2.0 ** (byte[:, i] - 127.0) for i in (0, 1))
    with np.errstate(over="ignore", under="ignore"):
        h = g / (1 + np.exp(-g)) * u
    assert np.isfinite(h).all()
    # silu: 2^-21 of itself, below -87 1.1e-36 in all; h in 8 bits: half a step, 2^-4 of itself, or 2^-10 of the least scale
    slack = 2.0 ** -21 * np.abs(h) + np.where(g < -87, 1.1e-36, 0) * np.abs(u)
    off = slack + 2.0 ** -4 * (np.abs(h) + slack) + 2.0 ** -136
    bad = ~(np.abs(out - h[:, None]) <= off[:, None])
    assert not bad.any(), [(g[t], u[t], h[t], out[t, 0]) for t in np.flatnonzero(bad.any(1))[:6]]
