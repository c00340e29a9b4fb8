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


# ---------------------------------------------------------------------------
# 4-bit weights at both ends of fp32
# ---------------------------------------------------------------------------
# Every kernel: a row of one and of several stages, few strips, whole k and parts of k.
W4_ENDS = [(1, 100, 300), (1, 40, 33000), (7, 33, 4095), (50, 31, 1023), (9, 900, 6001), (20, 500, 9000), (9, 8300, 130),
           (33, 8300, 31), (49, 8300, 65)]


def w4_ends_case(M, N, K, group, zeros, seed):
    """Codes, rows and zero points whose groups' sums have one sign, so that no sum passes the last:
    x, q, z, groups."""
    rng = np.random.default_rng(seed)
    groups = -(-K // group)
    x = rng.integers(0, 9, (M, K)).astype(np.int8)
    q = rng.integers(8, 16, (N, K)).astype(np.uint8)
    z = rng.integers(0, 9, (N, groups)).astype(np.uint8) if zeros else None
    return x, q, z, groups


def w4_ends_check(x, s_a, q, sc, z, group, dtype):
    """Sums that are exact in fp32 (below 33000 * 15 * 8 * 3 < 2^24 units, of one scale or three): the
    output is that sum times s_a, rounded once.  The product of 24 bits and 24 is exact in 64."""
    (M, K), N = x.shape, q.shape[0]
    assert sc.dtype == torch.float64 and torch.equal(sc.to(dtype).double(), sc)
    packed = w2a8.pack_w4a8(torch.from_numpy(block.w4_interchange(q)), sc.to(dtype), N, K, group,
                            None if z is None else torch.from_numpy(z)).to(dev())
    y, size = block.w4_product(x, np.ones(M), q, sc.numpy(), z, group)
    assert size.max() <= np.finfo(np.float32).max
    with np.errstate(over="ignore"):
        want = torch.from_numpy((y * s_a.astype(np.float64)[:, None]).astype(np.float32))
    f = torch.empty((M, N), device=dev())
    b = torch.empty((M, N), dtype=torch.bfloat16, device=dev())
    w2a8.w4a8_gemm(packed, torch.from_numpy(x).to(dev()), torch.from_numpy(s_a).to(dev()), M, N, K, group, dtype,
                   z is not None, f, b)
    torch.cuda.synchronize()
    assert torch.equal(f.cpu(), want)
    assert torch.equal(b.cpu(), want.bfloat16())
    return y, want


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", W4_ENDS)
def test_w4_smallest_token_scales(M, N, K, group, zeros, dtype):
    """Token scales down to the smallest subnormal keep all of their bits."""
    x, q, z, groups = w4_ends_case(M, N, K, group, zeros, M + N + K)
    rng = np.random.default_rng(K)
    sign = torch.from_numpy(rng.choice([-1.0, 1.0], (N, 1))).expand(N, groups).contiguous()
    ends = np.array([1.1e-38, 1e-40, 3e-42, 2.0 ** -149], np.float32)
    for i in range(4 if M == 1 else 1):
        w4_ends_check(x, ends[(np.arange(M) + i) % 4], q, sign, z, group, dtype)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", W4_ENDS)
def test_w4_sums_up_to_the_largest_value(M, N, K, group, zeros):
    """bf16 scales whose largest sum is in the top two powers of two of fp32."""
    x, q, z, groups = w4_ends_case(M, N, K, group, zeros, M + N + K + 1)
    rng = np.random.default_rng(K)
    sign = rng.choice([-1.0, 1.0], (N, 1)) * np.ones((N, groups))
    most = block.w4_product(x, np.ones(M), q, sign, z, group)[1].max()
    sc = torch.from_numpy(sign * 2.0 ** (128 - int(np.ceil(np.log2(most)) + (np.log2(most) % 1 == 0))))
    for s_a in (np.ones(M), rng.uniform(0.5, 1, M) * 2.0 ** -100):
        y, want = w4_ends_check(x, s_a.astype(np.float32), q, sc, z, group, torch.bfloat16)
        assert np.abs(y).max() >= 2.0 ** 126 and want.isfinite().all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", W4_ENDS)
def test_w4_smallest_group_scales(M, N, K, group, zeros, dtype):
    """One and three times the smallest subnormal of the scales' type."""
    x, q, z, groups = w4_ends_case(M, N, K, group, zeros, M + N + K + 2)
    rng = np.random.default_rng(K)
    sc = torch.from_numpy(rng.choice([1.0, 3.0], (N, groups)) * torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps)
    w4_ends_check(x, (rng.uniform(0.5, 1, M) * (2.0 ** 100 if dtype == torch.bfloat16 else 1)).astype(np.float32), q, sc, z, group,
                  dtype)


@pytest.mark.parametrize("H,I,E,top_k", [(48, 49152, 2, 1), (33, 24576, 3, 2), (33, 24577, 3, 2), (100, 2560, 10, 8), (100, 2561, 10, 8)])
def test_moe_one_token_round_the_border(H, I, E, top_k, kernels):
    """One token's longest hidden rows, both kernels: the reference's result, and the same bits."""
    c = Moe(1, H, I, E, H + I)
    got = w2a8.moe(*c.args(), H, I, top_k, "relu2")
    c.check(got, top_k, "relu2", True)
    for mode in (1, 2):
        kernels(mode)
        assert torch.equal(w2a8.moe(*c.args(), H, I, top_k, "relu2"), got)
