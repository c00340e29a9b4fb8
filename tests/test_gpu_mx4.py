"""GPU tests of the MX4 operators against the plain 64-bit reference.

Rounding, packing and reading back are exact: bytes and values are equal.

Products are tested twice.  With scale bytes 126..128 every product is a
multiple of 2^-4 (values are multiples of 1/2, scales at least 1/2 each), so
every partial sum is exact in fp32 as long as the sum of magnitudes stays
below 2^20 (24 bits above 2^-4), whatever the order: the outputs are equal to
the reference.  With scales spread over 2^-10..2^10, an output may be off by
the fp32 additions on its way: at most four blocks' sums per tile of 128 are
added into one accumulator, at most 8 waves' sums are joined, and s_w is
multiplied in once; each of these rounds or cuts off at most one unit 2^-23 of
a magnitude that the sum of magnitudes S bounds, so |error| <= (4 KT + 9) *
2^-23 * S.  A bf16 output is the fp32 one rounded half to even: equal bits.
"""
import threading

import numpy as np
import pytest
import torch

import w2a8_gemv_amd as w2a8
from oracle import mx4
from gpu_util import dev, packed_on_device, to_dev

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
GUARD = 64


def guarded_bytes(n):
    return torch.full((n + GUARD,), 0xA5, dtype=torch.uint8, device=dev())


def assert_guard_bytes(t, n):
    assert bool((t[n:] == 0xA5).all()), "write past the end"


def float_rows(R, K, seed, dtype):
    """Rows of mixed magnitude, as the type holds them; float64 values beside them."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((R, K)) * np.exp2(rng.integers(-6, 7, (R, -(-K // 16))).repeat(16, 1)[:, :K])
    x[rng.random((R, K)) < 0.1] = 0
    t = torch.from_numpy(x.astype(np.float32)).to(dtype)
    return t, t.double().numpy()


def mx_rows(R, K, seed, low=126, high=128):
    """Random codes and scale bytes (low..high)."""
    rng = np.random.default_rng(seed)
    return (rng.integers(0, 16, (R, K)).astype(np.uint8),
            rng.integers(low, high + 1, (R, -(-K // 32))).astype(np.uint8))


def on_device(codes, scales):
    q, s = mx4.rows_layout(codes, scales)
    return to_dev(q), to_dev(s)


# ---------------------------------------------------------------------------
# rounding and reading back
# ---------------------------------------------------------------------------
ROWS = [(1, 1), (1, 31), (2, 32), (3, 33), (1, 127), (5, 128), (2, 129), (3, 512), (2, 513),
        (7, 1000), (1, 2560), (19, 4095), (2, 4096), (2, 6907), (300, 65), (1, 27648)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,K", ROWS)
def test_quant_and_dequant_match_reference(M, K, dtype):
    x, x64 = float_rows(M, K, 7 * M + K, dtype)
    nq, ns = w2a8.mx4_act_bytes(M, K), w2a8.mx4_scale_bytes(M, K)
    q, s = guarded_bytes(nq), guarded_bytes(ns)
    w2a8.quant_act_mx4(x.to(dev()), q, s)
    torch.cuda.synchronize()
    codes, scales = mx4.quant(x64)
    want_q, want_s = mx4.rows_layout(codes, scales)
    np.testing.assert_array_equal(q[:nq].cpu().numpy(), want_q.reshape(-1))
    np.testing.assert_array_equal(s[:ns].cpu().numpy(), want_s.reshape(-1))
    assert_guard_bytes(q, nq)
    assert_guard_bytes(s, ns)
    y = torch.full((M * K + GUARD,), 77.0, dtype=dtype, device=dev())
    w2a8.dequant_act_mx4(q, s, K, M, dtype=dtype, y=y[:M * K])
    torch.cuda.synchronize()
    np.testing.assert_array_equal(y[:M * K].double().cpu().numpy().reshape(M, K),
                                  mx4.values(codes, scales))
    assert bool((y[M * K:] == 77.0).all())


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_quant_special_values(dtype):
    """Ties, saturation, signed zeros, subnormals, the type's largest values,
    not-a-numbers and infinities, in an even and an odd row length."""
    f = torch.finfo(dtype)
    for K in (256, 259):
        x = torch.zeros((12, K), dtype=dtype)
        ties = torch.tensor([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 5.125, 0.1875, 0.3125, -0.25,
                             -5, -1.75, -0.0, -0.3125], dtype=dtype)
        x[0, :16] = ties
        x[1, :16] = ties * 1.25                       # largest 7.5: saturates at 6
        x[2] = f.max
        x[3] = -f.max
        x[3, 5] = f.tiny
        x[4] = f.smallest_normal / 4                  # subnormal rows
        x[5] = torch.arange(K) % 7 * f.smallest_normal / 8
        x[6, 40] = float("nan")
        x[7, 255] = float("inf")
        x[8, 0] = -float("inf")
        x[9, K - 1] = 1.0
        x[10] = -0.0
        x[11] = torch.arange(K) - 100.0
        q, s = w2a8.quant_act_mx4(x.to(dev()))
        y = w2a8.dequant_act_mx4(q, s, K)
        torch.cuda.synchronize()
        codes, scales = mx4.quant(x.double().numpy())
        want_q, want_s = mx4.rows_layout(codes, scales)
        np.testing.assert_array_equal(q.cpu().numpy(), want_q)
        np.testing.assert_array_equal(s.cpu().numpy(), want_s)
        np.testing.assert_array_equal(y.cpu().numpy().astype(np.float64), mx4.values(codes, scales))
        assert np.isnan(y[6, 32:64].cpu().numpy()).all() and not y[6, :32].isnan().any()


def test_dequant_every_code_and_scale():
    """All 16 codes under all 256 scale bytes, in each type."""
    codes = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    scales = np.arange(256, dtype=np.uint8).reshape(256, 1)
    q, s = on_device(codes, scales)
    v = mx4.values(codes, scales)
    for dtype in TYPES:
        y = w2a8.dequant_act_mx4(q, s, 32, dtype=dtype)
        torch.cuda.synchronize()
        want = torch.from_numpy(v).float().to(dtype).double().numpy()   # v is exact in fp32
        np.testing.assert_array_equal(y.double().cpu().numpy(), want)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("N,K", [(1, 1), (15, 33), (16, 128), (17, 129), (100, 700), (33, 2560), (5, 6907)])
def test_quant_pack_matches_reference(N, K, dtype):
    W, w64 = float_rows(N, K, N + K, dtype)
    nb = w2a8.mx4_packed_bytes(N, K)
    p = guarded_bytes(nb)
    w2a8.quant_pack_mx4(W.to(dev()), packed=p)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(p[:nb].cpu().numpy(), mx4.packed_layout(*mx4.quant(w64)))
    assert_guard_bytes(p, nb)


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------
def weights(kind, N, K, seed, low=126, high=128):
    """(packed weights on the device, their float64 values [N, K])."""
    if kind == "w4":
        c, s = mx_rows(N, K, seed, low, high)
        return to_dev(mx4.packed_layout(c, s)), mx4.values(c, s)
    w = np.random.default_rng(seed).integers(-1, 2, (N, K)).astype(np.int8)
    return packed_on_device(w), w.astype(np.float64)


def gemm(kind, wp, q, s, M, N, K, s_w=1.0):
    """Both outputs of a product, each in front of a guard band."""
    yf = torch.full((M * N + GUARD,), 77.0, device=dev())
    yb = torch.full((M * N + GUARD,), 77.0, device=dev(), dtype=torch.bfloat16)
    if kind == "w4":
        w2a8.w4mx4_gemm(wp, q, s, M, N, K, yf[:M * N], yb[:M * N])
    else:
        w2a8.w2mx4_gemm(wp, q, s, M, N, K, s_w, yf[:M * N], yb[:M * N])
    torch.cuda.synchronize()
    assert bool((yf[M * N:] == 77).all()) and bool((yb[M * N:] == 77).all()), "write past the end"
    return yf[:M * N].view(M, N), yb[:M * N].view(M, N)


def assert_product(kind, M, N, K, seed, low=126, high=128, exact=True):
    c, s = mx_rows(M, K, seed, low, high)
    wp, w = weights(kind, N, K, seed + 1, low, high)
    s_w = 1.0 if kind == "w4" else 0.75 if exact else float(np.float32(0.0213))
    want, mag = mx4.product(mx4.values(c, s), w, s_w)
    yf, yb = gemm(kind, wp, *on_device(c, s), M, N, K, s_w)
    got = yf.cpu().numpy().astype(np.float64)
    if exact:
        # (times s_w = 3/4: two more bits)
        assert mag.max() < 2 ** 18
        np.testing.assert_array_equal(got, want)
    else:
        tol = (4 * -(-K // 128) + 9) * 2.0 ** -23 * mag
        assert (np.abs(got - want) <= tol).all(), np.abs((got - want) / tol).max()
    assert torch.equal(yb, yf.to(torch.bfloat16))


KINDS = ["w4", "w2"]
# one size for every output tile that the launch plans of 256 compute units
# choose among (rows x columns over k-groups), and the largest over several
# turns of the ring: 16 x 64 over 8, 32 x 64 over 4 (MX4) and 32 x 256
# (ternary), 64 x 64 and 32 x 128 over 4, 64 x 128 over 2, 32 x 256 (MX4), 64 x
# 256, 128 x 256, 256 x 256 (MX4) and 128 x 256 (ternary)
PLANS = [(74, 102, 2064), (36, 100, 130), (64, 100, 514), (2100, 235, 1048), (2052, 196, 523),
         (2084, 213, 137), (2083, 863, 132), (2105, 962, 132), (2071, 1812, 132), (2008, 6186, 133),
         (1967, 6454, 1100), (2157, 203, 1153)]
# the largest tiles with the other kind of result stores (whole lines or long k
# against large outputs of odd rows)
STORES = [(2574, 4672, 387), (3920, 1091, 128), (548, 7698, 133), (3277, 3712, 648), (1415, 5490, 129)]
# strips of weights as many as compute units, a few more and more than two for
# each, at the weight stream's two kinds of short batches; long k
STREAMS = [(1, 4096, 4100), (9, 4096, 4100), (24, 4096, 4100), (24, 4112, 3000), (32, 8200, 2100),
           (24, 8300, 1100), (17, 16500, 520), (16, 9000, 1030), (17, 4100, 20500), (20, 8200, 20480)]
# every edge of rows, columns and k: blocks of 32, tiles of 128, groups of 512
SMALL = [(1, 1, 1), (1, 16, 31), (2, 17, 32), (1, 33, 33), (3, 15, 127), (16, 16, 128), (17, 32, 129),
         (31, 100, 257), (33, 7, 384), (16, 48, 511), (1, 64, 512), (5, 65, 513), (64, 33, 640),
         (65, 96, 1000), (1, 100, 2560), (1, 31, 4097), (130, 257, 300), (19, 130, 1536)]
# odd and even sizes across the launch plans' rules
LARGE = [(1, 2560, 2560), (1, 5120, 6912), (1, 3000, 13825), (8, 2560, 2560), (16, 1111, 3200),
         (19, 3840, 2560), (32, 2500, 1280), (48, 1000, 2560), (64, 2560, 6912), (100, 1300, 1100),
         (128, 1024, 2560), (129, 515, 2561), (256, 1280, 700), (257, 2049, 260), (512, 2560, 640),
         (1000, 777, 1025), (2045, 300, 130)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,N,K", SMALL + LARGE + PLANS + STORES + STREAMS)
def test_product_is_exact(M, N, K, kind):
    assert_product(kind, M, N, K, seed=M + 3 * N + 5 * K)


@pytest.mark.parametrize("kind", KINDS)
def test_large_outputs_of_odd_rows(kind):
    """Outputs of more than 24 MiB whose rows are no whole lines, with a short k
    (every row of results equals that of a product of few rows)."""
    M, N, K = 1300, 6151, 100
    c, s = mx_rows(M, K, 8)
    wp, _ = weights(kind, N, K, 9)
    yf, yb = gemm(kind, wp, *on_device(c, s), M, N, K)
    for m in (0, 1, 640, 1277):
        f, b = gemm(kind, wp, *on_device(c[m:m + 23], s[m:m + 23]), 23, N, K)
        assert torch.equal(yf[m:m + 23], f) and torch.equal(yb[m:m + 23], b)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,N,K", [(1, 70, 2560), (1, 40, 27648), (7, 100, 1000), (16, 64, 6912),
                                   (33, 200, 2561), (128, 256, 2560), (300, 520, 1300)])
def test_product_of_spread_scales(M, N, K, kind):
    assert_product(kind, M, N, K, seed=M + N + K, low=117, high=137, exact=False)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M", [1, 5, 40, 200])
def test_nan_blocks_reach_their_rows_and_columns_only(M, kind):
    N, K = 50, 700
    c, s = mx_rows(M, K, 1)
    s[M - 1, 3] = 255
    w = np.random.default_rng(2).integers(-1, 2, (N, K)).astype(np.int8)
    if kind == "w4":
        wc, ws = mx_rows(N, K, 2)
        ws[7, -1] = 255
        wp = to_dev(mx4.packed_layout(wc, ws))
    else:
        wp = packed_on_device(w)
    yf, yb = gemm(kind, wp, *on_device(c, s), M, N, K)
    want = np.zeros((M, N), bool)
    want[M - 1] = True
    if kind == "w4":
        want[:, 7] = True
    np.testing.assert_array_equal(np.isnan(yf.cpu().numpy()), want)
    np.testing.assert_array_equal(np.isnan(yb.float().cpu().numpy()), want)


@pytest.mark.parametrize("M", [1, 20, 150])
def test_smallest_and_largest_scales(M):
    """2^-127 against large scales, results down to fp32's subnormals and up to
    infinity."""
    N, K = 40, 160
    for lx, hx, lw, hw in ((0, 2, 200, 203), (50, 52, 60, 62), (250, 252, 3, 5), (254, 254, 250, 252)):
        c, s = mx_rows(M, K, lx, lx, hx)
        wc, ws = mx_rows(N, K, lw, lw, hw)
        want, mag = mx4.product(mx4.values(c, s), mx4.values(wc, ws))
        yf, _ = gemm("w4", to_dev(mx4.packed_layout(wc, ws)), *on_device(c, s), M, N, K)
        got = yf.cpu().numpy().astype(np.float64)
        if lx == 254:      # every partial sum passes fp32's range or is far above 1
            assert (~np.isfinite(got) | (np.abs(got) > 1) | (want == 0)).all()
            continue
        # each rounding: 2^-23 of S, or half the smallest subnormal per block
        tol = 17 * 2.0 ** -23 * mag + 17 * 2.0 ** -149
        assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("kind", KINDS)
def test_one_output_and_outputs_of_both(kind):
    M, N, K = 5, 90, 300
    c, s = mx_rows(M, K, 3)
    q, sc = on_device(c, s)
    wp, _ = weights(kind, N, K, 4)
    yf, yb = gemm(kind, wp, q, sc, M, N, K)
    if kind == "w4":
        f, b = (w2a8.gemm_w4mx4(wp, q, sc, N, K, out_dtype=t) for t in (torch.float32, torch.bfloat16))
    else:
        f, b = (w2a8.gemm_w2mx4(wp, q, sc, 1.0, N, K, out_dtype=t) for t in (torch.float32, torch.bfloat16))
    assert torch.equal(f, yf) and torch.equal(b, yb)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,N,K", PLANS + [(1, 40, 300), (9, 90, 700), (29, 1000, 300)])
def test_each_output_alone_equals_both(M, N, K, kind):
    """A product into one of its outputs, at every output tile, from rows in a
    buffer made for more of them."""
    c, s = mx_rows(M + 3, K, 5)
    q, sc = on_device(c, s)
    wp, _ = weights(kind, N, K, 6)
    yf, yb = gemm(kind, wp, q, sc, M, N, K)
    f = torch.full((M, N), 77.0, device=dev())
    b = torch.full((M, N), 77.0, device=dev(), dtype=torch.bfloat16)
    for out in ({"y_f32": f}, {"y_bf16": b}):
        if kind == "w4":
            w2a8.w4mx4_gemm(wp, q, sc, M, N, K, **out)
        else:
            w2a8.w2mx4_gemm(wp, q, sc, M, N, K, 1.0, **out)
    torch.cuda.synchronize()
    assert torch.equal(f, yf) and torch.equal(b, yb)


# ---------------------------------------------------------------------------
# whole layers
# ---------------------------------------------------------------------------
def layer(kind, x, wp, N, K, **kw):
    return (w2a8.linear_w4mx4(x, wp, N, K, **kw) if kind == "w4"
            else w2a8.linear_w2mx4(x, wp, 0.375, N, K, **kw))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("N,K", [(1, 1), (16, 32), (33, 100), (40, 511), (100, 512), (48, 515), (2560, 2560),
                                 (130, 4100), (50, 27648), (3, 70001)])
def test_fused_layer_equals_the_two_steps(N, K, dtype, kind):
    x, x64 = float_rows(1, K, N + K, dtype)
    wp, w = weights(kind, N, K, 5)
    xd = x.to(dev())
    for out in (torch.float32, torch.bfloat16):
        y1 = layer(kind, xd, wp, N, K, out_dtype=out)
        y2 = layer(kind, xd, wp, N, K, out_dtype=out, fused=False)
        torch.cuda.synchronize()
        assert y1.dtype == out and y1.shape == (1, N) and torch.equal(y1, y2)
    s_w = 1.0 if kind == "w4" else 0.375
    want, mag = mx4.product(mx4.values(*mx4.quant(x64)), w, s_w)
    tol = (4 * -(-K // 128) + 9) * 2.0 ** -23 * mag
    got = layer(kind, xd, wp, N, K).double().cpu().numpy()
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("kind", KINDS)
def test_fused_layer_with_nan_and_special_rows(kind):
    N, K = 20, 600
    wp, w = weights(kind, N, K, 6)
    for at, v in ((599, float("nan")), (0, float("inf")), (300, 3e38), (511, 1e-40)):
        x = torch.zeros(K)
        x[at] = v
        y1 = layer(kind, x.to(dev()), wp, N, K)
        y2 = layer(kind, x.to(dev()), wp, N, K, fused=False)
        torch.cuda.synchronize()
        np.testing.assert_array_equal(y1.cpu().numpy(), y2.cpu().numpy())
        assert bool(y1.isnan().all()) == (not np.isfinite(v))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M", [1, 3, 33, 150])
def test_a_run_of_layers(M, kind):
    """Two layers behind each other, as a feed-forward block uses them, with
    weights rounded on the device."""
    H, I = 320, 850
    x, x64 = float_rows(M, H, 11, torch.bfloat16)
    if kind == "w4":
        up, up64 = float_rows(I, H, 12, torch.float32)
        down, down64 = float_rows(H, I, 13, torch.float32)
        pu, pd = w2a8.quant_pack_mx4(up.to(dev())), w2a8.quant_pack_mx4(down.to(dev()))
        wu, wd = mx4.values(*mx4.quant(up64)), mx4.values(*mx4.quant(down64))
        s_w = 1.0
    else:
        (pu, wu), (pd, wd), s_w = weights("w2", I, H, 12), weights("w2", H, I, 13), 0.375
    h = layer(kind, x.to(dev()), pu, I, H, out_dtype=torch.bfloat16)
    y = layer(kind, torch.relu(h).square(), pd, H, I)
    torch.cuda.synchronize()
    want_h, mag_h = mx4.product(mx4.values(*mx4.quant(x64)), wu, s_w)
    got_h = h.double().cpu().numpy()
    # the fp32 sum's bound, then half a step of bf16 of the result
    tol_h = (4 * 3 + 9) * 2.0 ** -23 * mag_h
    assert (np.abs(got_h - want_h) <= tol_h + 2.0 ** -8 * (np.abs(want_h) + tol_h)).all()
    a = torch.relu(h).square().double().cpu().numpy()          # the second layer's own input
    want, mag = mx4.product(mx4.values(*mx4.quant(a)), wd, s_w)
    assert (np.abs(y.double().cpu().numpy() - want) <= (4 * 7 + 9) * 2.0 ** -23 * mag).all()


# ---------------------------------------------------------------------------
# streams, graphs, refusals on the device
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M", [1, 24, 200])
def test_captured_layers_replay_like_eager_ones(M, kind):
    """Two graphs of the same call, replayed in turn with new inputs, eager
    calls between them."""
    N, K = 300, 1300
    wp, _ = weights(kind, N, K, 21)
    xs = [float_rows(M, K, 30 + i, torch.bfloat16)[0].to(dev()) for i in range(4)]
    want = [layer(kind, x, wp, N, K).clone() for x in xs]
    static = [x.clone() for x in xs[:2]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for x in static:
            layer(kind, x, wp, N, K)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for x in static:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(layer(kind, x, wp, N, K))
        graphs.append(g)
    for i in range(6):
        for j in range(2):
            static[j].copy_(xs[(i + j) % 4])
            graphs[j].replay()
        eager = layer(kind, xs[i % 4], wp, N, K)
        torch.cuda.synchronize()
        assert torch.equal(eager, want[i % 4])
        for j in range(2):
            assert torch.equal(outs[j], want[(i + j) % 4])


@pytest.mark.parametrize("kind", KINDS)
def test_calls_on_several_streams_at_once(kind):
    N, K = 500, 2560
    wp, _ = weights(kind, N, K, 22)
    Ms = [1, 9, 40, 140]
    xs = [float_rows(M, K, M, torch.float16)[0].to(dev()) for M in Ms]
    want = [layer(kind, x, wp, N, K) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in Ms]
    got = []
    for _ in range(5):
        for x, st in zip(xs, streams):
            got.append(layer(kind, x, wp, N, K, stream=st))
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 4])


def test_calls_from_several_host_threads():
    """Threads with streams of their own, each over all operators."""
    N, K = 300, 1000
    packed = {kind: weights(kind, N, K, 40)[0] for kind in KINDS}
    xs = [float_rows(M, K, 50 + M, torch.bfloat16)[0].to(dev()) for M in (1, 7, 50, 130)]
    want = [[layer(kind, x, packed[kind], N, K) for kind in KINDS] + [w2a8.quant_act_mx4(x)] for x in xs]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        st = torch.cuda.Stream()
        for _ in range(20):
            got = [layer(kind, xs[i], packed[kind], N, K, stream=st) for kind in KINDS]
            q, s = w2a8.quant_act_mx4(xs[i], stream=st)
            st.synchronize()
            same = [torch.equal(a, b) for a, b in zip(got + [q, s], want[i][:2] + list(want[i][2]))]
            if not all(same):
                wrong.append((i, same))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_outputs_over_inputs_are_refused():
    x = torch.ones((1, 64), device=dev())
    wp = w2a8.quant_pack_mx4(torch.ones((64, 64), device=dev()))
    wt = packed_on_device(np.ones((64, 64), np.int8))
    with pytest.raises(w2a8.W2A8Error):
        w2a8.w4mx4_linear_gemv(wp, x, 64, 64, y_f32=x)
    with pytest.raises(w2a8.W2A8Error):
        w2a8.w2mx4_linear_gemv(wt, x, 64, 64, y_f32=x)
    q, s = w2a8.quant_act_mx4(x)
    with pytest.raises(w2a8.W2A8Error):
        w2a8.dequant_act_mx4(q, s, 16, 1, y=q.view(torch.float32).view(-1)[:16])
    with pytest.raises(w2a8.W2A8Error):
        w2a8.quant_act_mx4(x, x.view(torch.uint8))
    torch.cuda.synchronize()
    assert bool((x == 1).all())


def test_device_refusals():
    x = torch.zeros((4, 64), device=dev())
    q, s = w2a8.quant_act_mx4(x)
    wp = w2a8.quant_pack_mx4(torch.zeros((16, 64), device=dev()))
    with pytest.raises(ValueError):
        w2a8.quant_act_mx4(x.t())                                   # not contiguous
    with pytest.raises(ValueError):
        w2a8.quant_act_mx4(x.view(1, 4, 64))
    with pytest.raises(w2a8.W2A8Error):
        w2a8.quant_act_mx4(x[:0])                                   # no rows
    with pytest.raises(w2a8.W2A8Error):
        w2a8.quant_act_mx4(x[:, :0].contiguous())
    with pytest.raises(w2a8.W2A8Error):
        w2a8.quant_act_mx4(x.view(-1)[1:65])                        # not 16-byte aligned
    with pytest.raises(ValueError):
        w2a8.quant_act_mx4(x, q[:3], s)                             # too small
    with pytest.raises(ValueError):
        w2a8.dequant_act_mx4(q, s.cpu(), 64)
    with pytest.raises(ValueError):
        w2a8.dequant_act_mx4(q, s, 640)
    with pytest.raises(TypeError):
        w2a8.dequant_act_mx4(q, s, 64, dtype=torch.float64)
    with pytest.raises(ValueError):
        w2a8.gemm_w4mx4(wp, q.view(-1), s, 16, 64)                  # rows not told
    with pytest.raises(ValueError):
        w2a8.gemm_w4mx4(wp[:-1], q, s, 16, 64)
    with pytest.raises(ValueError):
        w2a8.gemm_w2mx4(wp[:100], q, s, 1.0, 16, 64)
    with pytest.raises(TypeError):
        w2a8.gemm_w4mx4(wp, q, s, 16, 64, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        w2a8.w4mx4_gemm(wp, q, s, 4, 16, 64, y_f32=torch.empty(63, device=dev()))
    with pytest.raises(w2a8.W2A8Error):
        w2a8.w4mx4_gemm(wp, q, s, 4, 16, 64)                        # no output
    with pytest.raises(ValueError):
        w2a8.linear_w4mx4(x, wp, 16, 65)
    with pytest.raises(ValueError):
        w2a8.w4mx4_linear_gemv(wp, x, 16, 64, y_f32=torch.empty(16, device=dev()))


@pytest.mark.parametrize("kind", KINDS)
def test_rows_of_another_k_are_refused(kind):
    """Rows counted by their first dimension have to be rows of the K given;
    larger buffers are taken where M is given or, for scales, where flat."""
    M, N, K = 3, 40, 300
    c, s = mx_rows(M, 700, 70)
    wp, _ = weights(kind, N, K, 71)
    long_q, long_s = on_device(c, s)
    q, sc = on_device(c[:, :K], s[:, :10])
    call = lambda a, b: (w2a8.gemm_w4mx4(wp, a, b, N, K) if kind == "w4"
                         else w2a8.gemm_w2mx4(wp, a, b, 1.0, N, K))
    for a, b in ((long_q, long_s), (long_q, sc), (q, long_s)):
        with pytest.raises(ValueError):
            call(a, b)
        with pytest.raises(ValueError):
            w2a8.dequant_act_mx4(a, b, K)
    want, _ = gemm(kind, wp, q, sc, M, N, K)
    flat = torch.cat([sc.view(-1), torch.zeros(64, dtype=torch.uint8, device=dev())])
    more = torch.cat([sc, sc])
    for b in (sc, flat, more):
        assert torch.equal(call(q, b), want)
    values = w2a8.dequant_act_mx4(q, sc, K)
    assert torch.equal(w2a8.dequant_act_mx4(torch.cat([q, q]).view(-1), flat, K, M), values)
    assert torch.equal(w2a8.dequant_act_mx4(q, flat, K), values)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M", [1, 20, 150])
def test_single_products_at_the_ends_of_fp32(M, kind):
    """One product of other than 0 to each output: products of 4-bit values
    (multiples of 1/4, at most six bits) are exact from the smallest subnormal
    up to fp32's largest value; from 2^128 on they are infinities of their
    sign.  (A value below 2^128 of six bits is below fp32's largest.)"""
    N, K = 40, 160
    rng = np.random.default_rng(M)
    c = np.zeros((M, K), np.uint8)
    c[np.arange(M), 7 * np.arange(M) % K] = rng.integers(0, 16, M)
    scale_pairs = (((254, 250), (254, 128), (252, 127), (190, 191), (27, 80), (0, 107)) if kind == "w4"
                   else ((254, 127), (253, 127), (251, 127), (0, 127), (1, 127)))
    for sx, sw in scale_pairs:
        s = np.full((M, 5), sx, np.uint8)
        if kind == "w4":
            wc = rng.integers(0, 16, (N, K)).astype(np.uint8)
            ws = np.full((N, 5), sw, np.uint8)
            wp, w = to_dev(mx4.packed_layout(wc, ws)), mx4.values(wc, ws)
        else:
            wp, w = weights(kind, N, K, 9)
        want = mx4.values(c, s) @ w.T
        assert ((np.abs(want) >= 2.0 ** 128) | (np.abs(want) <= np.finfo(np.float32).max)).all()
        with np.errstate(over="ignore"):
            want = torch.from_numpy(want.astype(np.float32)).to(dev())
        yf, yb = gemm(kind, wp, *on_device(c, s), M, N, K)
        assert torch.equal(yf, want), (sx, sw)
        assert torch.equal(yb, want.to(torch.bfloat16)), (sx, sw)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M", [1, 20, 150])
def test_sums_past_fp32_are_infinities_of_their_sign(M, kind):
    """Products of one sign, each below fp32's largest value, the sum above it."""
    N, K = 40, 1000
    sign = np.arange(M)[:, None] % 2
    c = np.broadcast_to(2 + 8 * sign, (M, K)).astype(np.uint8)           # 1 and -1
    s = np.full((M, -(-K // 32)), 254, np.uint8)                        # 2^127
    wc, ws = np.full((N, K), 2, np.uint8), np.full((N, -(-K // 32)), 127, np.uint8)
    wp = (to_dev(mx4.packed_layout(wc, ws)) if kind == "w4"
          else packed_on_device(np.ones((N, K), np.int8)))
    yf, yb = gemm(kind, wp, *on_device(c, s), M, N, K)
    want = torch.where(torch.from_numpy(sign == 1), -float("inf"), float("inf")).to(dev()).expand(M, N)
    assert torch.equal(yf, want) and torch.equal(yb.float(), want)
