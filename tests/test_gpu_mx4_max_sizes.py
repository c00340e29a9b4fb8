"""GPU tests of the MX4 operators at their size limits and past 2^31 bytes.

Inputs hold values whose products are known without a reference product."""
import pytest
import torch

import w2a8_gemv_amd as w2a8
from gpu_util import dev

pytestmark = pytest.mark.gpu

KMAX = 1048448


def ones_rows(M, K, value=1.0):
    return w2a8.quant_act_mx4(torch.full((M, K), value, device=dev()))


@pytest.mark.parametrize("M", [1, 3, 40])
def test_longest_k(M):
    """K at its limit: every output is the sum of K ones (exact: below 2^24)."""
    N = 33
    x = torch.full((M, KMAX), 1.0, device=dev(), dtype=torch.bfloat16)
    wp = w2a8.quant_pack_mx4(torch.full((N, KMAX), 1.0, device=dev(), dtype=torch.bfloat16))
    wt = w2a8.pack_ternary(torch.ones((N, KMAX), dtype=torch.int8)).to(dev())
    for y in (w2a8.linear_w4mx4(x, wp, N, KMAX), w2a8.linear_w2mx4(x, wt, 0.5, N, KMAX) * 2):
        assert bool((y == KMAX).all())
    q, s = w2a8.quant_act_mx4(x)
    assert bool((w2a8.dequant_act_mx4(q, s, KMAX, dtype=torch.bfloat16) == 1).all())


def test_weights_past_4_gib():
    """MX4 and ternary weights of more than 2^32 bytes: the last rows, which a
    32-bit offset would miss, hold values of their own."""
    K, N = 4096, (1 << 21) + 24 * 1024 + 5
    assert w2a8.mx4_packed_bytes(N, K) > (1 << 32)
    W = torch.zeros((N, K), device=dev(), dtype=torch.bfloat16)
    W[-1] = 3.0
    W[1 << 20, ::2] = -1.0
    wp = w2a8.quant_pack_mx4(W)
    del W
    want = torch.zeros(N, device=dev())
    want[-1] = 3.0 * K
    want[1 << 20] = -K / 2
    for M in (1, 20):
        y = w2a8.gemm_w4mx4(wp, *ones_rows(M, K), N, K)
        assert torch.equal(y, want.expand(M, N))
    del wp, y
    # ternary: a strip is 32 rows, codes of weight 0 are 01
    Nt = (1 << 22) + 40 * 1024
    assert w2a8.packed_bytes(Nt, K) > (1 << 32)
    wt = torch.full((w2a8.packed_bytes(Nt, K),), 0x55, dtype=torch.uint8, device=dev())
    wt[-1024 * (K // 128):] = 0xAA                      # the last strip: all weights 1
    for M in (1, 20):
        y = w2a8.gemm_w2mx4(wt, *ones_rows(M, K), 1.0, Nt, K)
        assert bool((y[:, -32:] == K).all()) and not bool(y[:, :-32].any())


def test_rows_past_4_gib():
    """Rows whose codes pass 2^32 bytes (and values 2^34): the last ones are read
    and written."""
    M, K = 1 << 20, 8200
    x = torch.zeros((M, K), device=dev(), dtype=torch.bfloat16)
    x[-1] = 2.0
    x[M // 2, :100] = 1.0
    q, s = w2a8.quant_act_mx4(x)
    assert q.numel() > (1 << 32)
    back = w2a8.dequant_act_mx4(q, s, K, dtype=torch.bfloat16)
    assert torch.equal(back, x)
    del back, x
    N = 5
    wp = w2a8.quant_pack_mx4(torch.ones((N, K), device=dev()))
    y = w2a8.gemm_w4mx4(wp, q, s, N, K)
    want = torch.zeros((M, N), device=dev())
    want[-1] = 2.0 * K
    want[M // 2] = 100.0
    assert torch.equal(y, want)


def test_outputs_past_2_to_31_elements():
    M, N, K = 40000, 60000, 32
    x = torch.zeros((M, K), device=dev())
    x[-1] = 1.0
    x[100, 0] = 4.0
    q, s = w2a8.quant_act_mx4(x)
    wp = w2a8.quant_pack_mx4(torch.ones((N, K), device=dev()))
    wt = w2a8.pack_ternary(torch.ones((N, K), dtype=torch.int8)).to(dev())
    for y in (w2a8.gemm_w4mx4(wp, q, s, N, K, out_dtype=torch.bfloat16),
              w2a8.gemm_w2mx4(wt, q, s, 1.0, N, K, out_dtype=torch.bfloat16)):
        assert bool((y[-1] == 32).all()) and bool((y[100] == 4).all())
        assert not bool(y[:100].any()) and not bool(y[101:-1].any())


def test_most_strips():
    """More strips than a grid's first dimension takes."""
    K, N = 32, (1 << 25) + 3                            # ternary strips of 32 rows
    wt = torch.full((w2a8.packed_bytes(N, K),), 0x55, dtype=torch.uint8, device=dev())
    wt[-1024:] = 0xAA
    y = w2a8.gemm_w2mx4(wt, *ones_rows(1, K), 1.0, N, K)
    assert bool((y[0, 1 << 25:] == 32).all()) and not bool(y[0, :1 << 25].any())
    N = (1 << 24) + 3                                   # MX4 strips of 16
    wp = torch.zeros(w2a8.mx4_packed_bytes(N, K), dtype=torch.uint8, device=dev())
    tile = w2a8.pack_mx4(torch.full((16, K // 2), 0x22, dtype=torch.uint8),
                         torch.full((16, 1), 127, dtype=torch.uint8), 16, K).to(dev())
    strips = (1 << 20) + 1
    wp[(strips - 1) * 1024:strips * 1024] = tile[:1024]
    wp[-256:] = tile[1024:]
    y = w2a8.gemm_w4mx4(wp, *ones_rows(1, K), N, K)
    assert bool((y[0, 1 << 24:] == 32).all()) and not bool(y[0, :1 << 24].any())
