"""GPU tests of the operators around the ternary layers at the ends of their
types' ranges, against the plain 64-bit reference."""
import numpy as np
import pytest
import torch

import w2a8_gemv_amd as w2a8
from oracle import block
from gpu_util import dev
from test_gpu_block import UNIT, Moe

pytestmark = pytest.mark.gpu


@pytest.fixture
def kernels():
    """Sets the kernels of the mixture, and the automatic choice afterwards."""
    yield w2a8.tune_moe
    w2a8.tune_moe(0)


# ---------------------------------------------------------------------------
# mixture of experts: an expert whose scale is broken
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf, 3e38, -3e38], ids=str)
@pytest.mark.parametrize("which", ["gate", "up", "down"])
@pytest.mark.parametrize("act", ["relu2", "silu"])
@pytest.mark.parametrize("mode", [1, 2, 4])
def test_moe_broken_expert_marks_its_tokens_alone(mode, act, which, value, kernels):
    """NaN and infinity appear where the reference has them (a gate that is not a number, or passes
    the range to either side, is never lost), and tokens that do not take the expert do not notice.
    Hidden rows of one value, so that nothing else of the row marks it, and of many."""
    kernels(mode)
    for I in (1, 70):
        M, H, E, top_k, spoilt = 20, 96, 6, 2, 3
        c = Moe(M, H, I, E, 9)
        good = w2a8.moe(*c.args(), H, I, top_k, act)
        c.s[["gate", "up", "down"].index(which)][spoilt] = value
        got = w2a8.moe(*c.args(), H, I, top_k, act)
        torch.cuda.synchronize()
        l = c.logits.float().double().numpy()
        takes = np.array([any(e == spoilt for e, _ in route) for route in block.moe_route(l, top_k, True)])
        assert takes.any() and not takes.all()
        assert torch.equal(got[torch.from_numpy(~takes)], good[torch.from_numpy(~takes)])
        with np.errstate(all="ignore"):
            want, bound = block.moe(c.x, c.s_a, l, *c.w, *c.s, top_k, act, True)
            bound = bound + (40 + 2 * top_k) * UNIT * c.magnitudes(l, top_k, act, True) + 1e-37
            want = np.where(np.abs(want) > np.finfo(np.float32).max, np.sign(want) * np.inf, want)
        got = got.double().cpu().numpy()
        np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
        np.testing.assert_array_equal(got[np.isinf(want)], want[np.isinf(want)])
        fine = np.isfinite(want)
        assert (np.abs(got[fine] - want[fine]) <= bound[fine]).all()
        if not np.isfinite(value) and which != "down":
            assert np.isnan(got[takes]).all()
