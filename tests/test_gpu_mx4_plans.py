"""GPU tests of every kernel that the MX4 products choose among, at sizes whose
k comes round its ring several times (mx4_sizes.py).  Values and scales are
those of the exact products of test_gpu_mx4.py: outputs equal the 64-bit
reference, whatever the order of the sums."""
import numpy as np
import pytest
import torch

import mx4_sizes
import w2a8_gemv_amd as w2a8
from gpu_util import dev
from oracle import mx4
from test_gpu_mx4 import GUARD, mx_rows, on_device, weights

pytestmark = pytest.mark.gpu

SIZES = [(kind,) + size for kind in ("w4", "w2")
         for size in mx4_sizes.ROUNDS[kind] + mx4_sizes.STAY[kind] + mx4_sizes.STREAM[kind]]


@pytest.mark.parametrize("kind,M,N,K", SIZES)
def test_every_plan_and_selection_of_outputs_is_exact(kind, M, N, K):
    c, s = mx_rows(M, K, M + K)
    q, sc = on_device(c, s)
    wp, w = weights(kind, N, K, N + K)
    s_w = 1.0 if kind == "w4" else 0.75
    want, mag = mx4.product(mx4.values(c, s), w, s_w)
    assert mag.max() < 2 ** 18                   # every partial sum is exact in fp32
    want = torch.from_numpy(want.astype(np.float32)).to(dev())
    for f32, bf16 in ((True, False), (False, True), (True, True)):
        yf = torch.full((M * N + GUARD,), 77.0, device=dev()) if f32 else None
        yb = torch.full((M * N + GUARD,), 77.0, device=dev(), dtype=torch.bfloat16) if bf16 else None
        out = {"y_f32": yf[:M * N] if f32 else None, "y_bf16": yb[:M * N] if bf16 else None}
        if kind == "w4":
            w2a8.w4mx4_gemm(wp, q, sc, M, N, K, **out)
        else:
            w2a8.w2mx4_gemm(wp, q, sc, M, N, K, s_w, **out)
        torch.cuda.synchronize()
        if f32:
            assert torch.equal(yf[:M * N].view(M, N), want)
            assert bool((yf[M * N:] == 77).all()), "write past the end"
        if bf16:
            assert torch.equal(yb[:M * N].view(M, N), want.to(torch.bfloat16))
            assert bool((yb[M * N:] == 77).all()), "write past the end"
