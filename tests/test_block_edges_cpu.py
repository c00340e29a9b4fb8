"""CPU tests of the operators around the ternary layers: calls that fit the
documented types and sizes, but not the buffers that they come with."""
import numpy as np
import pytest
import torch

import w2a8_gemv_amd as w2a8


def test_w4_unpacking_refuses_weights_of_another_form():
    """Weights packed with zero points do not come back without them, nor those of one group as
    another's: the buffer has to be exactly the form's."""
    rng = np.random.default_rng(0)
    N, K = 20, 300
    codes = torch.from_numpy(rng.integers(0, 256, (N, K // 2)).astype(np.uint8))
    for group in (32, 64, 128):
        shape = (N, -(-K // group))
        scales = torch.from_numpy(rng.uniform(0.5, 2, shape)).half()
        for z in (None, torch.from_numpy(rng.integers(0, 16, shape).astype(np.uint8))):
            p = w2a8.pack_w4a8(codes, scales, N, K, group, z)
            c, s, back = w2a8.unpack_w4a8(p, N, K, group, zeros=z is not None)
            assert torch.equal(c, codes) and torch.equal(s, scales) and (z is None or torch.equal(back, z))
            with pytest.raises((ValueError, w2a8.W2A8Error)):
                w2a8.unpack_w4a8(p, N, K, group, zeros=z is None)
            with pytest.raises(ValueError):
                w2a8.unpack_w4a8(torch.cat([p, p[:16]]), N, K, group, zeros=z is not None)
            for other in {32, 64, 128} - {group}:
                with pytest.raises((ValueError, w2a8.W2A8Error)):
                    w2a8.unpack_w4a8(p, N, K, other, zeros=z is not None)


def test_moe_plan_of_one_token():
    """One or two experts go by themselves as long as their hidden rows fit LDS; of more, fewer
    workgroups the more maxima each has to take.  The border is where it is for any device."""
    one = lambda I, E, top_k, cus=256: w2a8.moe_plan(1, 2048, I, E, top_k, cus)[0] == 1  # noqa: E731
    for I in (32736, 32768, 40960, 49152):
        assert one(I, 8, 1) and one(I // 2, 8, 2)
    assert not one(49153, 8, 1) and not one(24577, 8, 2)
    for cus in (64, 256, 304):
        for top_k in (3, 4, 8, 12, 16):
            most = 40 * cus // (top_k + 8)                   # workgroups: strips of 32 times top_k
            assert one(32 * (most // top_k), 16, top_k, cus)
            assert not one(32 * (most // top_k) + 1, 16, top_k, cus)
