"""GPU tests of the norm into int8 rows, the products with 4-bit weights and the
mixture of ternary experts, against the plain 64-bit reference.

Norm: codes and h are equal; the scale is rounded once from a value whose sum
in fp64 may have been added in another order, so it may be the neighbouring
fp32: one unit 2^-23 of itself.

4-bit weights: a group's sum is an exact integer.  With scales 0.5, 1 and 2 and
a token scale of 1 every term is a multiple of 1/2, and with at most 2000 columns
the sum of magnitudes is below 2000 * 15 * 127 * 2 < 2^23: outputs are equal.
Otherwise each group's multiply-add, each join and the token scale round once,
by at most 2^-24 of the magnitudes summed so far.  Waves hold disjoint groups,
so their multiply-adds cost at most groups * S in all, S the sum of the groups'
magnitudes; one row joins up to 8 waves (7 S), more rows up to 4 groups of waves
(3 S) and then 8 parts of k (7 S): |error| <= (groups + 11) * 2^-24 * S.  A bf16 output is the
fp32 one rounded half to even: equal bits.

Mixture: every step to the experts' outputs is stated in fp32 and equal to the
reference's for relu2 (for silu: the reference's bound).  A weight p is off by
the exponential (2 units of 2^-24 and its argument's rounding, at most 20 units
for arguments above -20; smaller weights count nothing), at most 256 additions
in trees of at most 16 levels, and a division: 40 units; an output by its top_k
products and additions: |error| <= (40 + 2 top_k) * 2^-24 * sum |p part|.
"""
import threading

import numpy as np
import pytest
import torch

import block_sizes
import w2a8_gemv_amd as w2a8
from oracle import block
from gpu_util import dev, packed_on_device

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
UNIT = 2.0 ** -24
GUARD = 64


def guarded(n, dtype, fill=77):
    return torch.full((n + GUARD,), fill, dtype=dtype, device=dev())


def assert_guard(t, n, fill=77):
    assert bool((t[n:] == fill).all()), "write past the end"


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------
def norm_inputs(M, K, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(M, K, generator=g) * 0.5).to(dtype)
    r = (torch.randn(M, K, generator=g) * torch.where(torch.rand(K, generator=g) < 0.02, 20.0, 1.0)).to(dtype)
    w = (1 + 0.2 * torch.randn(K, generator=g)).to(dtype)
    return x, r, w


def norm_check(x, r, w, eps, q, s, h, **kw):
    want_h = x if r is None else (x.float() + r.float()).to(x.dtype)
    codes, scale = block.rmsnorm_quant(want_h.double().numpy(), None if w is None else w.double().numpy(), eps)
    np.testing.assert_array_equal(q.cpu().numpy(), codes)
    got = s.double().cpu().numpy()
    np.testing.assert_array_equal(np.isnan(got), np.isnan(scale))
    fine = ~np.isnan(scale)
    assert (np.abs(got - scale)[fine] <= 2.0 ** -23 * scale[fine]).all()
    if h is not None:
        torch.testing.assert_close(h.cpu(), want_h, rtol=0, atol=0, equal_nan=True)


NORM = [(1, 1), (2, 7), (1, 8), (3, 9), (2, 63), (5, 64), (1, 513), (4, 2560), (3, 6907), (2, 8192), (2, 8193), (1, 16385),
        (2, 24577), (1, 32768), (2, 32769), (1, 40008), (700, 65)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,K", NORM)
def test_norm_matches_reference(M, K, dtype):
    x, r, w = norm_inputs(M, K, dtype, 3 * M + K)
    for residual, weight, eps in ((r, w, 1e-5), (None, w, 0.0), (r, None, 1e-6), (None, None, 1.0)):
        q, s, h = guarded(M * K, torch.int8), guarded(M, torch.float32), guarded(M * K, dtype)
        d = lambda t: None if t is None else t.to(dev())
        xd = d(x)
        out = w2a8.rmsnorm_quant_int8(xd, d(weight), d(residual), eps, q[:M * K].view(M, K), s[:M],
                                      None if residual is None else h[:M * K].view(M, K))
        torch.cuda.synchronize()
        assert_guard(q, M * K), assert_guard(s, M), assert_guard(h, M * K)
        assert residual is not None or (out[2] is xd and bool((h == 77).all()))
        norm_check(x, residual, weight, float(np.float32(eps)), out[0], out[1], None if residual is None else out[2])


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("K", [1, 3, 7, 8, 9, 10, 12, 14, 15, 17, 20, 23, 511, 513, 519, 1283, 1284, 4095, 8191, 8197, 32767,
                               32775, 32776, 32777])
def test_norm_rows_begin_anywhere(K, dtype):
    """Nine rows of each length begin at every place that it allows, and write no byte of another."""
    M = 9
    x, r, w = norm_inputs(M, K, dtype, K)
    q, s, h = guarded(M * K, torch.int8), guarded(M, torch.float32), guarded(M * K, dtype)
    out = w2a8.rmsnorm_quant_int8(x.to(dev()), w.to(dev()), r.to(dev()), 1e-5, q[:M * K].view(M, K), s[:M], h[:M * K].view(M, K))
    torch.cuda.synchronize()
    assert_guard(q, M * K), assert_guard(s, M), assert_guard(h, M * K)
    norm_check(x, r, w, float(np.float32(1e-5)), *out)
    rd = r.to(dev())
    again = w2a8.rmsnorm_quant_int8(x.to(dev()), w.to(dev()), rd, 1e-5, h=rd)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, again))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("K", [2048, 2049, 4096, 4097, 5123, 6144, 6151, 8192, 8201, 16390, 24583])
def test_norm_of_more_rows_than_compute_units(K, dtype):
    """Every count of chunks a lane, with and without ends."""
    M = 300
    x, r, w = norm_inputs(M, K, dtype, K)
    for residual in (r, None):
        out = w2a8.rmsnorm_quant_int8(x.to(dev()), w.to(dev()), None if residual is None else r.to(dev()), 1e-5)
        torch.cuda.synchronize()
        norm_check(x, residual, w, float(np.float32(1e-5)), *out)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("K", [40, 1003, 33001])
def test_norm_in_place(K, dtype):
    x, r, w = norm_inputs(3, K, dtype, K)
    for which in ("residual", "x"):
        xd, rd = x.to(dev()), r.to(dev())
        q, s, h = w2a8.rmsnorm_quant_int8(xd, w.to(dev()), rd, 1e-5, h=rd if which == "residual" else xd)
        torch.cuda.synchronize()
        norm_check(x, r, w, float(np.float32(1e-5)), q, s, h)
        assert torch.equal((xd if which == "residual" else rd).cpu(), x if which == "residual" else r)
    xd = x.to(dev())
    q, s, h = w2a8.rmsnorm_quant_int8(xd, None, xd, 1e-5, h=xd)         # one buffer for all three
    torch.cuda.synchronize()
    norm_check(x, x, None, float(np.float32(1e-5)), q, s, h)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("K", [48, 333, 32775])
def test_norm_special_rows(K, dtype):
    """Zero rows, subnormal ones, ties, the type's largest values, NaN and infinities."""
    f = torch.finfo(dtype)
    x = torch.zeros((10, K), dtype=dtype)
    x[1] = f.smallest_normal / 4
    x[2] = f.max
    x[3] = -f.max
    x[3, 1] = f.tiny
    x[4, K - 1] = float("nan")
    x[5, 0] = float("inf")
    x[6, 3] = -float("inf")
    x[7] = ((torch.arange(K) % 254) / 2 - 63.5).to(dtype)
    x[7, 0] = 127.0                                                    # codes of half values: ties
    x[8, K - 1] = -1.0
    x[9] = -0.0
    for r in (None, x.flip(0).contiguous(), x):
        for w in (None, torch.full((K,), 3.0, dtype=dtype), torch.zeros(K, dtype=dtype)):
            d = lambda t: None if t is None else t.to(dev())
            q, s, h = w2a8.rmsnorm_quant_int8(d(x), d(w), d(r), 0.0)
            torch.cuda.synchronize()
            norm_check(x, r, w, 0.0, q, s, h if r is not None else None)


def test_norm_feeds_the_ternary_product():
    """The rows are those that the products take: exact integers."""
    x, r, w = norm_inputs(3, 640, torch.bfloat16, 1)
    q, s, h = w2a8.rmsnorm_quant_int8(x.to(dev()), w.to(dev()), r.to(dev()))
    wt = np.random.default_rng(0).integers(-1, 2, (100, 640)).astype(np.int8)
    y_i32, y = w2a8.gemm(packed_on_device(wt), q, 100, 640, s_a=s, s_w=0.5)
    torch.cuda.synchronize()
    acc = q.cpu().numpy().astype(np.int64) @ wt.T.astype(np.int64)
    np.testing.assert_array_equal(y_i32.cpu().numpy(), acc)
    np.testing.assert_array_equal(y.cpu().numpy(), acc.astype(np.float32) * s.cpu().numpy()[:, None] * np.float32(0.5))


# ---------------------------------------------------------------------------
# 4-bit weights
# ---------------------------------------------------------------------------
def w4_case(M, N, K, group, zeros, dtype, seed, exact):
    rng = np.random.default_rng(seed)
    groups = -(-K // group)
    x = rng.integers(-127, 128, (M, K)).astype(np.int8)
    x[rng.random((M, K)) < 0.05] = -127
    if exact == "small":
        x = rng.integers(-8, 9, (M, K)).astype(np.int8)
    q = rng.integers(0, 16, (N, K)).astype(np.uint8)
    z = rng.integers(0, 16, (N, groups)).astype(np.uint8) if zeros else None
    if exact:
        most = [0.5, 1.0] if exact == "small" else [0.5, 1.0, 2.0]
        s_a, sc = np.ones(M, np.float32), rng.choice(most, (N, groups)) * rng.choice([-1, 1], (N, groups))
    else:
        s_a = rng.uniform(0.001, 0.1, M).astype(np.float32)
        sc = rng.uniform(0.001, 0.02, (N, groups)) * 2.0 ** rng.integers(-6, 7, (N, groups))
    sc = torch.from_numpy(sc).to(dtype)
    zt = None if z is None else torch.from_numpy(z)
    packed = w2a8.pack_w4a8(torch.from_numpy(block.w4_interchange(q)), sc, N, K, group, zt).to(dev())
    y, size = block.w4_product(x, s_a, q, sc.double().numpy(), z, group)
    return torch.from_numpy(x).to(dev()), torch.from_numpy(s_a).to(dev()), packed, y, size, groups


def w4_run(M, N, K, group, zeros, dtype, seed, exact, stream=None):
    x, s_a, packed, y, size, groups = w4_case(M, N, K, group, zeros, dtype, seed, exact)
    f, b = guarded(M * N, torch.float32), guarded(M * N, torch.bfloat16)
    w2a8.w4a8_gemm(packed, x, s_a, M, N, K, group, dtype, zeros, f[:M * N], b[:M * N])
    torch.cuda.synchronize()
    assert_guard(f, M * N), assert_guard(b, M * N)
    got = f[:M * N].cpu()
    assert torch.equal(b[:M * N].cpu(), got.bfloat16())
    got = got.double().numpy().reshape(M, N)
    if exact:
        np.testing.assert_array_equal(got, y)
    else:
        assert (np.abs(got - y) <= (groups + 11) * UNIT * size + 1e-37).all()
    for one, dt in ((f, torch.float32), (b, torch.bfloat16)):       # one output alone
        alone = w2a8.gemm_w4a8(packed, x, s_a, N, K, group, dtype, zeros, dt)
        torch.cuda.synchronize()
        assert torch.equal(alone.flatten(), one[:M * N])


W4_KN = [(1, 1), (31, 5), (32, 16), (33, 17), (64, 40), (96, 15), (127, 33), (128, 16), (129, 100), (256, 64), (300, 31),
         (513, 48), (1000, 90), (1999, 20)]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 32, 33, 64])
def test_w4_exact_sums(M, group, zeros):
    for K, N in W4_KN:
        w4_run(M, N, K, group, zeros, torch.float16 if (K + M) % 2 else torch.bfloat16, K + N + M, True)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("M,N,K,group,zeros", [
    (1, 2560, 2560, 128, False), (1, 640, 6912, 64, True), (1, 300, 27648, 32, False), (3, 1000, 2570, 32, True),
    (16, 500, 5120, 128, True), (19, 700, 2561, 64, False), (31, 333, 6907, 32, False), (47, 200, 4096, 128, False),
    (64, 256, 8640, 64, True), (64, 1030, 1280, 32, True), (1, 9000, 640, 128, False), (40, 9000, 129, 32, True)])
def test_w4_rounded_sums(M, N, K, group, zeros, dtype):
    w4_run(M, N, K, group, zeros, dtype, M + N + K, False)


@pytest.mark.parametrize("M,N,K", [size for sizes in block_sizes.W4.values() for size in sizes])
def test_w4_every_plan_is_exact(M, N, K):
    """Rows of -8..8: sums of magnitudes below 66001 * 15 * 8 * 1 < 2^23, in units of 1/2."""
    for i, (group, zeros) in enumerate(((32, True), (64, False), (128, True))):
        w4_run(M, N, K, group, zeros, (torch.float16, torch.bfloat16)[(i + K) % 2], M + N + K + i, "small")


def test_w4_extreme_values():
    """All codes and rows at their ends: the largest sums of a group."""
    for group in (32, 64, 128):
        for zeros in (None, 0, 15):
            for code in (0, 15):
                N, K, M = 16, 256, 17
                x = np.full((M, K), -127, np.int8)
                q, z = np.full((N, K), code, np.uint8), None
                if zeros is not None:
                    z = np.full((N, K // group), zeros, np.uint8)
                sc = torch.full((N, K // group), 1.0, dtype=torch.float16)
                p = w2a8.pack_w4a8(torch.from_numpy(block.w4_interchange(q)), sc, N, K, group,
                                   None if z is None else torch.from_numpy(z)).to(dev())
                y = w2a8.gemm_w4a8(p, torch.from_numpy(x).to(dev()), torch.ones(M, device=dev()), N, K, group,
                                   zeros=z is not None)
                torch.cuda.synchronize()
                want = -127 * K * (code - (8 if zeros is None else zeros))
                assert bool((y == want).all())


def test_w4_special_scales_stay_in_their_rows():
    """A NaN, infinite or zero group scale or token scale marks its own outputs alone."""
    M, N, K, group = 5, 40, 300, 64
    rng = np.random.default_rng(2)
    q = rng.integers(0, 16, (N, K)).astype(np.uint8)
    sc = torch.full((N, -(-K // group)), 0.5, dtype=torch.float16)
    sc[3, 1], sc[17, 4], sc[20] = float("nan"), float("inf"), 0
    p = w2a8.pack_w4a8(torch.from_numpy(block.w4_interchange(q)), sc, N, K, group).to(dev())
    x = torch.from_numpy(rng.integers(1, 128, (M, K)).astype(np.int8)).to(dev())
    sa = torch.ones(M, device=dev())
    sa[2] = float("nan")
    y = w2a8.gemm_w4a8(p, x, sa, N, K, group).cpu()
    assert y[:, 3].isnan().all() and not y[[0, 1, 3, 4], 17].isfinite().any() and (y[[0, 1, 3, 4], 20] == 0).all()
    assert y[2].isnan().all()
    rest = [n for n in range(N) if n not in (3, 17)]
    assert y[[0, 1, 3, 4]][:, rest].isfinite().all()


def test_linear_w4a8_is_quantizer_and_product():
    x = torch.randn(4, 200, generator=torch.Generator().manual_seed(1)).bfloat16().to(dev())
    q, s_a = w2a8.quant_act_int8(x)
    rng = np.random.default_rng(3)
    w = rng.integers(0, 16, (50, 200)).astype(np.uint8)
    sc = torch.from_numpy(rng.uniform(0.01, 0.02, (50, 2))).half()
    p = w2a8.pack_w4a8(torch.from_numpy(block.w4_interchange(w)), sc, 50, 200, 128).to(dev())
    assert torch.equal(w2a8.linear_w4a8(x, p, 50, 200, 128), w2a8.gemm_w4a8(p, q, s_a, 50, 200, 128))
    one = w2a8.linear_w4a8(x[0], p, 50, 200, 128, out_dtype=torch.bfloat16)
    assert torch.equal(one[0], w2a8.gemm_w4a8(p, q[0], s_a[:1], 50, 200, 128)[0].bfloat16())


# ---------------------------------------------------------------------------
# mixture of experts
# ---------------------------------------------------------------------------
class Moe:
    def __init__(self, M, H, I, E, seed):
        rng = np.random.default_rng(seed)
        self.M, self.H, self.I, self.E = M, H, I, E
        self.x = rng.integers(-127, 128, (M, H)).astype(np.int8)
        self.s_a = rng.uniform(0.005, 0.05, M).astype(np.float32)
        self.w = [rng.integers(-1, 2, (E, n, k)).astype(np.int8) for n, k in ((I, H), (I, H), (H, I))]
        self.s = [rng.uniform(0.5, 2, E).astype(np.float32) / np.float32(np.sqrt(k)) for k in (H, H, I)]
        self.logits = torch.from_numpy(2 * rng.standard_normal((M, E)))
        self.packed = [torch.stack([w2a8.pack_ternary(torch.from_numpy(w[e])) for e in range(E)]).to(dev()) for w in self.w]
        self.rows = torch.from_numpy(self.x).to(dev())

    def args(self, logits=None, dtype=torch.float32, x=None, s_a=None):
        t = lambda a: torch.from_numpy(a).to(dev())
        return (self.rows if x is None else x, t(self.s_a) if s_a is None else s_a,
                (self.logits if logits is None else logits).to(dtype).to(dev()), *self.packed, *[t(s) for s in self.s])

    def check(self, got, top_k, act, renorm, logits=None, dtype=torch.float32, s_a=None):
        l = (self.logits if logits is None else logits).to(dtype).double().numpy()
        want, bound = block.moe(self.x, self.s_a if s_a is None else s_a, l, *self.w, *self.s, top_k, act, renorm)
        size = self.magnitudes(l, top_k, act, renorm, s_a)
        got = got.double().cpu().numpy()
        np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
        fine = ~np.isnan(want)
        assert (np.abs(got - want)[fine] <= (bound + (40 + 2 * top_k) * UNIT * size + 1e-37)[fine]).all()

    def magnitudes(self, l, top_k, act, renorm, s_a=None):
        """sum |p part| of every output, from one expert at a time."""
        total = np.zeros((self.M, self.H))
        for e in range(self.E):
            route = block.moe_route(l, top_k, renorm)
            p = np.array([0.0 if c is None else dict(c).get(e, 0.0) for c in route])
            rows = np.nonzero(p)[0]
            if len(rows):
                one, _ = block.moe(self.x[rows], (self.s_a if s_a is None else s_a)[rows], np.zeros((len(rows), 1)),
                                   *[w[e:e + 1] for w in self.w], *[s[e:e + 1] for s in self.s], 1, act, True)
                total[rows] += p[rows, None] * np.abs(one)
        return total


MOE = [  # M, H, I, E, top_k
    (1, 1, 1, 1, 1), (1, 33, 31, 3, 2), (2, 128, 128, 4, 4), (3, 129, 65, 2, 1), (15, 200, 96, 5, 3), (16, 256, 300, 8, 2),
    (17, 100, 130, 1, 1), (33, 64, 257, 2, 2), (64, 48, 40, 3, 2), (64, 32, 32, 256, 16), (7, 513, 127, 70, 9),
    (1, 640, 1000, 64, 8), (5, 1000, 1283, 6, 2), (64, 320, 700, 4, 2)]


@pytest.fixture
def kernels():
    """Sets the kernels of the mixture, and the automatic choice afterwards."""
    yield w2a8.tune_moe
    w2a8.tune_moe(0)


@pytest.mark.parametrize("mode", [0, 1, 3, 4])
@pytest.mark.parametrize("act", ["relu2", "silu"])
@pytest.mark.parametrize("M,H,I,E,top_k", MOE)
def test_moe_matches_reference(M, H, I, E, top_k, act, mode, kernels):
    kernels(mode)
    c = Moe(M, H, I, E, M + H + I)
    for renorm, dtype in ((True, torch.float32), (False, torch.bfloat16), (True, torch.float16)):
        f, b = guarded(M * H, torch.float32), guarded(M * H, torch.bfloat16)
        need = w2a8.w2a8_moe_workspace_bytes(M, H, I, E, top_k)
        ws = guarded(need, torch.uint8, 0xA5)
        w2a8.w2a8_moe(*c.args(dtype=dtype), M, H, I, E, top_k, act, renorm, f[:M * H], b[:M * H], ws[:need])
        torch.cuda.synchronize()
        assert_guard(f, M * H), assert_guard(b, M * H), assert_guard(ws, need, 0xA5)
        assert torch.equal(b[:M * H], f[:M * H].bfloat16())
        c.check(f[:M * H].view(M, H), top_k, act, renorm, dtype=dtype)
        for dt, one in ((torch.float32, f), (torch.bfloat16, b)):
            alone = w2a8.moe(*c.args(dtype=dtype), H, I, top_k, act, renorm, dt)
            assert torch.equal(alone.flatten(), one[:M * H])


@pytest.mark.parametrize("M,H,I,E,top_k", [size for sizes in block_sizes.MOE.values() for size in sizes])
def test_moe_every_plan(M, H, I, E, top_k):
    c = Moe(M, H, I, E, M + H + I)
    y = w2a8.moe(*c.args(), H, I, top_k, "relu2", True)
    c.check(y, top_k, "relu2", True)


@pytest.mark.parametrize("mode", [1, 2])
@pytest.mark.parametrize("renorm", [True, False])
def test_moe_masked_and_broken_logits(renorm, mode, kernels):
    """Masked experts are never taken, a token with none gives 0, NaN and infinity give NaN rows, ties
    go to the lower index, and the other tokens do not notice."""
    kernels(mode)
    inf, nan = float("inf"), float("nan")
    c = Moe(9, 96, 64, 70, 5)
    l = c.logits.clone()
    l[0] = -inf
    l[1] = -inf
    l[1, 69] = -3.0
    l[2, 10] = nan
    l[3, 68] = inf
    l[4] = 0.0
    l[5, ::2] = -inf
    l[6] = torch.where(torch.arange(70) % 2 == 0, 0.0, -0.0)
    l[7] = -3.0e38
    l[7, 3] = 3.0e38
    for dtype in (torch.float32, torch.bfloat16):
        y = w2a8.moe(*c.args(l, dtype), 96, 64, 3, "relu2", renorm)
        torch.cuda.synchronize()
        c.check(y, 3, "relu2", renorm, l, dtype)
        y = y.cpu()
        assert not y[0].any() and y[2].isnan().all() and y[3].isnan().all()


@pytest.mark.parametrize("mode", [1, 2])
def test_moe_broken_rows_stay_apart(mode, kernels):
    """A row whose scale is not finite, and one whose hidden values pass fp32, give NaN rows alone."""
    kernels(mode)
    c = Moe(4, 128, 64, 3, 8)
    s_a = c.s_a.copy()
    s_a[1], s_a[2] = np.nan, 1e30
    for act in ("relu2", "silu"):
        y = w2a8.moe(*c.args(s_a=torch.from_numpy(s_a).to(dev())), 128, 64, 2, act).cpu()
        assert y[1].isnan().all()
        assert y[[0, 3]].isfinite().all()
        good = w2a8.moe(*c.args(), 128, 64, 2, act).cpu()
        assert torch.equal(y[[0, 3]], good[[0, 3]])
        assert y[2].isnan().all()


@pytest.mark.parametrize("mode", [1, 2, 4])
def test_moe_zero_rows_and_one_expert(mode, kernels):
    kernels(mode)
    c = Moe(3, 256, 96, 2, 4)
    c.x[1] = 0
    c.rows = torch.from_numpy(c.x).to(dev())
    y = w2a8.moe(*c.args(), 256, 96, 2, "relu2")
    c.check(y, 2, "relu2", True)
    assert not y[1].any()
    # all tokens to one expert
    c = Moe(64, 256, 96, 5, 6)
    l = torch.zeros(64, 5)
    l[:, 3] = 5
    y = w2a8.moe(*c.args(l), 256, 96, 1, "silu")
    c.check(y, 1, "silu", True, l)


# ---------------------------------------------------------------------------
# together, captured, on other streams
# ---------------------------------------------------------------------------
class Block:
    """A block's feed-forward part and the head behind it, as one decode step runs them."""

    def __init__(self, M, seed):
        rng = np.random.default_rng(seed)
        self.c = Moe(M, 256, 160, 8, seed)          # (one token at a time; `kernels` for the others)
        g = torch.Generator().manual_seed(seed)
        self.x = torch.randn(M, 256, generator=g).bfloat16().to(dev())
        self.r = torch.randn(M, 256, generator=g).bfloat16().to(dev())
        self.w = [torch.rand(256, generator=g).add(0.5).bfloat16().to(dev()) for _ in range(2)]
        self.router, self.head = [self.pack(rng, n) for n in (8, 500)]

    @staticmethod
    def pack(rng, n):
        q = torch.from_numpy(block.w4_interchange(rng.integers(0, 16, (n, 256)).astype(np.uint8)))
        sc = torch.from_numpy(rng.uniform(0.001, 0.01, (n, 4))).half()
        return w2a8.pack_w4a8(q, sc, n, 256, 64).to(dev())

    def step(self, x, r):
        x_q, s_a, h = w2a8.rmsnorm_quant_int8(x, self.w[0], r)
        logits = w2a8.gemm_w4a8(self.router, x_q, s_a, 8, 256, 64)
        y = w2a8.moe(x_q, s_a, logits, *self.packed, 256, 160, 2, "relu2", out_dtype=torch.bfloat16)
        x_q, s_a, h = w2a8.rmsnorm_quant_int8(y, self.w[1], h)
        return w2a8.gemm_w4a8(self.head, x_q, s_a, 500, 256, 64), h, logits

    @property
    def packed(self):
        if not hasattr(self, "_packed"):
            self._packed = self.c.args()[3:]
        return self._packed


def test_block_together_matches_reference():
    """Each step of the run against the reference on the step's own inputs."""
    b = Block(5, 11)
    x_q, s_a, h = w2a8.rmsnorm_quant_int8(b.x, b.w[0], b.r)
    norm_check(b.x.cpu(), b.r.cpu(), b.w[0].cpu(), float(np.float32(1e-5)), x_q, s_a, h)
    out, h2, logits = b.step(b.x, b.r)
    y = w2a8.moe(x_q, s_a, logits, *b.packed, 256, 160, 2, "relu2")
    b.c.x, b.c.s_a = x_q.cpu().numpy(), s_a.cpu().numpy()
    b.c.check(y, 2, "relu2", True, logits.cpu())
    x2, s2, h3 = w2a8.rmsnorm_quant_int8(y.bfloat16(), b.w[1], h)
    norm_check(y.bfloat16().cpu(), h.cpu(), b.w[1].cpu(), float(np.float32(1e-5)), x2, s2, h3)
    assert torch.equal(h3, h2)
    assert torch.equal(out, w2a8.gemm_w4a8(b.head, x2, s2, 500, 256, 64))


@pytest.mark.parametrize("mode", [0, 2])
def test_two_graphs_replayed_between_eager_calls(mode, kernels):
    """Two captured steps, replayed with new inputs among eager work; every replay is equal to the
    eager result."""
    kernels(mode)
    blocks = [Block(1, 21), Block(19, 22)]
    graphs = []
    for b in blocks:
        b.step(b.x, b.r)                                           # (sizes and attributes are looked up once)
        b.gx, b.gr = b.x.clone(), b.r.clone()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.out = b.step(b.gx, b.gr)
        graphs.append(g)
    for i in range(4):
        for b, g in zip(blocks, graphs):
            b.gx.copy_(b.x * (i + 1) + i)
            b.gr.copy_(b.r - i)
            want = [t.clone() for t in b.step(b.gx, b.gr)]
            for t in b.out:
                t.fill_(-1)
            g.replay()
            torch.cuda.synchronize()
            for got, w in zip(b.out, want):
                assert torch.equal(got, w)


@pytest.mark.parametrize("mode", [0, 2])
def test_other_streams_and_threads(mode, kernels):
    """Steps on streams of their own, from host threads of their own."""
    kernels(mode)
    blocks = [Block(m, 30 + m) for m in (1, 7, 40)]
    want = [[t.clone() for t in b.step(b.x, b.r)] for b in blocks]
    torch.cuda.synchronize()
    bad = []

    def work(b, w):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                got = b.step(b.x, b.r)
                s.synchronize()
                bad.extend(i for i, (x, y) in enumerate(zip(got, w)) if not torch.equal(x, y))
    threads = [threading.Thread(target=work, args=a) for a in zip(blocks, want)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad


def test_stream_argument():
    b = Block(3, 41)
    want = b.step(b.x, b.r)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    x_q, s_a, h = w2a8.rmsnorm_quant_int8(b.x, b.w[0], b.r, stream=s)
    logits = w2a8.gemm_w4a8(b.router, x_q, s_a, 8, 256, 64, stream=s)
    y = w2a8.moe(x_q, s_a, logits, *b.packed, 256, 160, 2, "relu2", out_dtype=torch.bfloat16, stream=s)
    x_q, s_a, h = w2a8.rmsnorm_quant_int8(y, b.w[1], h, stream=s)
    got = w2a8.gemm_w4a8(b.head, x_q, s_a, 500, 256, 64, stream=s)
    s.synchronize()
    assert torch.equal(got, want[0]) and torch.equal(h, want[1])


@pytest.mark.parametrize("mode", [0, 2])
def test_repeated_calls_are_equal(mode, kernels):
    """Results do not depend on timing."""
    kernels(mode)
    b = Block(33, 51)
    want = [t.clone() for t in b.step(b.x, b.r)]
    for _ in range(30):
        for got, w in zip(b.step(b.x, b.r), want):
            assert torch.equal(got, w)


# ---------------------------------------------------------------------------
# offsets past 32 bits
# ---------------------------------------------------------------------------
def test_norm_past_32_bits():
    """2^20 rows of 2050: the last ones are those of a call on them alone (whose sum may round
    another way)."""
    x = torch.empty((1 << 20, 2050), dtype=torch.bfloat16, device=dev()).normal_()
    w = torch.rand(2050, device=dev()).bfloat16()
    q, s_a, _ = w2a8.rmsnorm_quant_int8(x, w)
    few = x[-300:].clone()
    qf, sf, _ = w2a8.rmsnorm_quant_int8(few, w)
    torch.cuda.synchronize()
    assert torch.equal(q[-300:], qf)
    assert ((s_a[-300:] - sf).abs() <= 2 * UNIT * sf).all()


@pytest.mark.parametrize("M", [1, 5, 40])
def test_w4_past_32_bits(M):
    """More than 2^31 bytes of codes: the last strips are those of a call on them alone.  Scales of
    1 and rows of -1..1 make every sum an exact one (below 16384 * 8 < 2^24)."""
    N, K = 264_000, 16384
    tiles = N // 16 * (K // 128) * 1024
    total = w2a8.w4a8_packed_bytes(N, K, 128)
    assert tiles > 2 ** 31
    p = torch.randint(0, 256, (total,), dtype=torch.uint8, device=dev())
    p[tiles:].view(torch.int16).fill_(0x3C00)
    x = torch.randint(-1, 2, (M, K), dtype=torch.int8, device=dev())
    s_a = torch.ones(M, device=dev())
    y = w2a8.gemm_w4a8(p, x, s_a, N, K, 128)
    n = 160
    last = torch.cat([p[tiles - n * K // 2:tiles], p[-2 * n * K // 128:]])
    part = w2a8.gemm_w4a8(last, x, s_a, n, K, 128)
    torch.cuda.synchronize()
    assert torch.equal(y[:, -n:], part) and part.abs().max() > 0


@pytest.mark.parametrize("M", [1, 40])
def test_moe_past_32_bits(M):
    """The last of 256 experts, past 2^31 bytes of each of the matrices, is the one of a call with
    it alone."""
    H, I, E = 5120, 6912, 256
    c = Moe(1, H, I, 1, 3)
    x = torch.randint(-127, 128, (M, H), dtype=torch.int8, device=dev())
    s_a, one = torch.full((M,), 0.01, device=dev()), torch.zeros((M, 1), device=dev())
    scales = [torch.from_numpy(s).to(dev()) for s in c.s]
    want = w2a8.moe(x, s_a, one, *c.packed, *scales, H, I, 1)
    all_w = [torch.full((E, w.numel()), 0x55, dtype=torch.uint8, device=dev()) for w in c.packed]   # (weights 0)
    for w, last in zip(all_w, c.packed):
        w[-1] = last[0]
    assert all_w[0].numel() > 2 ** 31 and all_w[2].numel() > 2 ** 31
    logits = torch.full((M, E), -1.0, device=dev())
    logits[:, -1] = 1.0
    got = w2a8.moe(x, s_a, logits, *all_w, *[s.expand(E).contiguous() for s in scales], H, I, 1)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and want.abs().max() > 0
