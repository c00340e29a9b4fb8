"""CPU tests of the MX4 operators: the reference's rounding on worked values,
the host packers and size queries against it, and the refusals of every entry
point (rejected before any HIP call: the stand-in pointers are never read)."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import mx4_sizes
import w2a8_gemv_amd as w2a8
from conftest import ROOT
from oracle import mx4

NULL, SHAPE, ALIGN, VALUE, BUFSIZE = 1, 2, 3, 4, 5
F = ctypes.c_float
FAKE = 0x10000


# ---------------------------------------------------------------------------
# the reference itself
# ---------------------------------------------------------------------------
def test_reference_rounding_of_worked_values():
    # one block whose largest magnitude is 6 (e = 0): ties go to even codes
    x = np.array([[6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 5.1, 0.2, 0.3, -0.25, -5, -1.75, 0, -0.3]])
    c, s = mx4.quant(x)
    assert s.tolist() == [[127]]
    assert mx4.values(c, s)[0].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, 6, 0, 0.5, 0, -4, -2, 0, -0.5]
    assert c[0, 11] == 8                               # a negative tie to zero keeps its sign
    # a = 7.9: e = 0, saturates at 6; a = 8: e = 1
    c, s = mx4.quant(np.array([[7.9]]))
    assert (c.tolist(), s.tolist()) == ([[7]], [[127]])
    c, s = mx4.quant(np.array([[8.0]]))
    assert (c.tolist(), s.tolist()) == ([[6]], [[128]])
    # zeros, the smallest exponent, not-a-numbers
    assert mx4.quant(np.zeros((1, 3)))[1].tolist() == [[0]]
    c, s = mx4.quant(np.array([[2.0 ** -127, 2.0 ** -128, 2.0 ** -130]]))
    assert (c.tolist(), s.tolist()) == ([[2, 1, 0]], [[0]])
    for bad in (np.nan, np.inf, -np.inf):
        c, s = mx4.quant(np.array([[1.0, bad] + [1.0] * 31]))
        assert s.tolist() == [[255, 125]] and not c[0, :32].any() and c[0, 32] == 6
        assert np.isnan(mx4.values(c, s)[0, :32]).all()


def test_reference_rounding_is_nearest():
    """At most half a step off (2^-2 of the value between 1 and 6 units), and
    idempotent."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((50, 320)) * np.exp2(rng.integers(-20, 20, (50, 1)))
    c, s = mx4.quant(x)
    v = mx4.values(c, s)
    unit = np.repeat(mx4.scale_values(s), 32, 1)
    y, m = np.abs(x) / unit, np.abs(v) / unit
    step = np.where(y < 2, 0.5, np.where(y < 4, 1, 2))
    assert (np.abs(y - m) <= np.where(y > 6, 2, step / 2)).all()
    # (a block whose largest value saturated or rounded down keeps its unit)
    c2, s2 = mx4.quant(v)
    np.testing.assert_array_equal(mx4.values(c2, s2), v)


# ---------------------------------------------------------------------------
# sizes and host packers
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("R,K", [(1, 1), (3, 31), (16, 128), (17, 129), (33, 512), (5, 513), (40, 2560)])
def test_sizes_and_packers_match_the_reference(R, K):
    rng = np.random.default_rng(R * K)
    codes = rng.integers(0, 16, (R, K)).astype(np.uint8)
    scales = rng.integers(0, 256, (R, -(-K // 32))).astype(np.uint8)
    q, s = mx4.rows_layout(codes, scales)
    assert w2a8.mx4_act_bytes(R, K) == q.size and w2a8.mx4_scale_bytes(R, K) == s.size
    inter = torch.from_numpy(mx4.interchange(codes))
    packed = w2a8.pack_mx4(inter, torch.from_numpy(scales), R, K)
    want = mx4.packed_layout(codes, scales)
    assert packed.numel() == want.size == w2a8.mx4_packed_bytes(R, K)
    np.testing.assert_array_equal(packed.numpy(), want)
    c, sc = w2a8.unpack_mx4(packed, R, K)
    np.testing.assert_array_equal(c.numpy(), inter.numpy())
    np.testing.assert_array_equal(sc.numpy(), scales)


def test_size_queries_refuse():
    L = w2a8.lib()
    for f in (L.mx4_act_bytes, L.mx4_scale_bytes, L.mx4_packed_bytes):
        assert f(0, 5) == -1 and f(5, 0) == -1 and f(5, 1048449) == -1 and f(5, 1048448) > 0
    assert L.mx4_act_bytes((1 << 20) + 1, 5) == -1 and L.mx4_packed_bytes((1 << 30) + 1, 5) == -1
    for f in (w2a8.mx4_act_bytes, w2a8.mx4_scale_bytes, w2a8.mx4_packed_bytes):
        with pytest.raises(w2a8.W2A8Error) as e:
            f(0, 16)
        assert e.value.status == SHAPE


def test_packers_refuse():
    L = w2a8.lib()
    c, s = np.zeros((4, 20), np.uint8), np.zeros((4, 2), np.uint8)
    out = np.zeros(w2a8.mx4_packed_bytes(4, 40), np.uint8)
    cp, sp, op, n = c.ctypes.data, s.ctypes.data, out.ctypes.data, out.size
    for args in ((None, sp, 4, 40, op, n), (cp, None, 4, 40, op, n), (cp, sp, 4, 40, None, n)):
        assert L.pack_mx4(*args) == NULL
    assert L.pack_mx4(cp, sp, 0, 40, op, n) == SHAPE
    assert L.pack_mx4(cp, sp, 4, 40, op, n - 1) == BUFSIZE
    assert L.pack_mx4(cp, sp, 4, 40, op, n) == 0
    assert L.unpack_mx4(op, n - 1, 4, 40, cp, sp) == BUFSIZE
    assert L.unpack_mx4(op, n, 4, 0, cp, sp) == SHAPE
    assert L.unpack_mx4(None, n, 4, 40, cp, sp) == NULL
    t = torch.zeros
    with pytest.raises(ValueError):
        w2a8.pack_mx4(t((4, 19), dtype=torch.uint8), t((4, 2), dtype=torch.uint8), 4, 40)
    with pytest.raises(ValueError):
        w2a8.pack_mx4(t((4, 20), dtype=torch.uint8), t((4, 1), dtype=torch.uint8), 4, 40)
    with pytest.raises(TypeError):
        w2a8.pack_mx4(t((4, 20)), t((4, 2), dtype=torch.uint8), 4, 40)
    with pytest.raises(w2a8.W2A8Error):
        w2a8.unpack_mx4(t(n - 1, dtype=torch.uint8), 4, 40)


# ---------------------------------------------------------------------------
# refusals of the device entry points
# ---------------------------------------------------------------------------
def test_row_entry_points_refuse():
    L = w2a8.lib()
    q = lambda x=FAKE, t=1, M=3, K=40, xq=FAKE, xs=FAKE: L.quant_act_mx4(x, t, M, K, xq, xs, None)
    d = lambda y=FAKE, t=1, M=3, K=40, xq=FAKE, xs=FAKE: L.dequant_act_mx4(xq, xs, M, K, y, t, None)
    for f, first in ((q, "x"), (d, "y")):
        assert f(**{first: None}) == NULL and f(xq=None) == NULL and f(xs=None) == NULL
        assert f(M=0) == SHAPE and f(K=0) == SHAPE and f(K=1048449) == SHAPE
        assert f(M=(1 << 20) + 1) == SHAPE
        assert f(t=-1) == VALUE and f(t=3) == VALUE
        assert f(**{first: FAKE + 2}) == ALIGN and f(xq=FAKE + 8) == ALIGN and f(xs=FAKE + 4) == ALIGN
    need = w2a8.mx4_packed_bytes(20, 300)
    p = lambda W=FAKE, t=0, N=20, K=300, o=FAKE, n=need: L.quant_pack_mx4(W, t, N, K, o, n, None)
    assert p(W=None) == NULL and p(o=None) == NULL and p(N=0) == SHAPE and p(t=7) == VALUE
    assert p(W=FAKE + 4) == ALIGN and p(o=FAKE + 8) == ALIGN and p(n=need - 1) == BUFSIZE


@pytest.mark.parametrize("kind", ["w4mx4", "w2mx4"])
def test_products_refuse(kind):
    L = w2a8.lib()
    sw = (F(1.0),) if kind == "w2mx4" else ()

    def g(w=FAKE, xq=FAKE, xs=FAKE, M=3, N=40, K=200, yf=FAKE, yb=FAKE):
        return getattr(L, kind + "_gemm")(w, xq, xs, M, N, K, *sw, yf, yb, None)

    def v(w=FAKE, x=FAKE, t=1, N=40, K=200, yf=FAKE, yb=FAKE):
        return getattr(L, kind + "_linear_gemv")(w, x, t, N, K, *sw, yf, yb, None)
    for f in (g, v):
        assert f(w=None) == NULL and f(yf=None, yb=None) == NULL
        assert f(N=0) == SHAPE and f(K=0) == SHAPE and f(N=(1 << 30) + 1) == SHAPE
        assert f(K=1048449) == SHAPE
        assert f(w=FAKE + 8) == ALIGN and f(yf=FAKE + 4) == ALIGN and f(yb=FAKE + 2) == ALIGN
    assert g(xq=None) == NULL and g(xs=None) == NULL and g(M=0) == SHAPE
    assert g(M=(1 << 20) + 1) == SHAPE and g(xq=FAKE + 8) == ALIGN and g(xs=FAKE + 4) == ALIGN
    assert v(x=None) == NULL and v(x=FAKE + 2) == ALIGN
    assert v(t=-1) == VALUE and v(t=3) == VALUE


def test_outputs_that_share_bytes_with_another_buffer_are_refused():
    """Each output against each other buffer of its call: over its first and
    its last 16 bytes."""
    L = w2a8.lib()
    M, N, K = 3, 40, 200
    at = {}

    def placed(sizes, out, other):
        """Buffers far apart, but `out` begins in the last 16 bytes of `other`."""
        for i, n in enumerate(sizes):
            at[n] = 0x1000000 * (i + 1)
        first = dict(at, **{out: at[other] + (sizes[other] - 1) // 16 * 16})
        last = dict(at, **{other: at[out] + (sizes[out] - 1) // 16 * 16})
        return first, last

    nq, ns = w2a8.mx4_act_bytes(M, K), w2a8.mx4_scale_bytes(M, K)
    for t, e in ((0, 4), (1, 2), (2, 2)):
        rows = {"x": M * K * e, "q": nq, "s": ns}
        for out, other in (("q", "x"), ("s", "x"), ("q", "s")):
            for b in placed(rows, out, other):
                assert L.quant_act_mx4(b["x"], t, M, K, b["q"], b["s"], None) == VALUE
        for other in "qs":
            for b in placed(rows, "x", other):
                assert L.dequant_act_mx4(b["q"], b["s"], M, K, b["x"], t, None) == VALUE
        nb = w2a8.mx4_packed_bytes(N, K)
        for b in placed({"W": N * K * e, "p": nb}, "p", "W"):
            assert L.quant_pack_mx4(b["W"], t, N, K, b["p"], nb, None) == VALUE
    for kind, nw in (("w4mx4", w2a8.mx4_packed_bytes(N, K)), ("w2mx4", w2a8.packed_bytes(N, K))):
        sw = (F(1.0),) if kind == "w2mx4" else ()
        sizes = {"w": nw, "q": nq, "s": ns, "f": M * N * 4, "b": M * N * 2}
        for out, other in (("f", "w"), ("f", "q"), ("f", "s"), ("b", "w"), ("b", "q"), ("b", "s"), ("f", "b")):
            for b in placed(sizes, out, other):
                assert getattr(L, kind + "_gemm")(b["w"], b["q"], b["s"], M, N, K, *sw, b["f"], b["b"],
                                                  None) == VALUE
        sizes = {"w": nw, "x": K * 4, "f": N * 4, "b": N * 2}
        for out, other in (("f", "w"), ("f", "x"), ("b", "w"), ("b", "x"), ("f", "b")):
            for b in placed(sizes, out, other):
                assert getattr(L, kind + "_linear_gemv")(b["w"], b["x"], 0, N, K, *sw, b["f"], b["b"],
                                                         None) == VALUE


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    u8 = torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(ValueError):
        w2a8.quant_act_mx4(x)
    with pytest.raises(ValueError):
        w2a8.linear_w4mx4(x, u8, 16, 64)
    with pytest.raises(ValueError):
        w2a8.linear_w2mx4(x, u8, 1.0, 16, 64)
    with pytest.raises(ValueError):
        w2a8.gemm_w4mx4(u8, u8.view(2, -1), u8, 16, 64)
    with pytest.raises(ValueError):
        w2a8.quant_pack_mx4(x.float())
    with pytest.raises(TypeError):
        w2a8.quant_act_mx4(x.double())
    with pytest.raises(TypeError):
        w2a8.quant_act_mx4([1.0])


def test_binding_refuses_rows_of_another_k(monkeypatch):
    """Rows of a longer K are a larger buffer, so their bytes alone do not tell
    them from rows of this one (refused before the library is called)."""
    monkeypatch.setattr(w2a8, "_mx4_gpu", lambda t, name: t.get_device())
    u8 = torch.uint8
    M, N, K = 3, 16, 64
    w = torch.zeros(w2a8.mx4_packed_bytes(N, K), dtype=u8)
    t = torch.zeros(w2a8.packed_bytes(N, K), dtype=u8)
    rows = lambda k: (torch.zeros((M, w2a8.mx4_act_bytes(1, k)), dtype=u8),
                      torch.zeros((M, w2a8.mx4_scale_bytes(1, k)), dtype=u8))
    q, s = rows(K)
    for k in (256, 640):                       # other codes; other codes and scales
        q2, s2 = rows(k)
        pairs = [(q2, s2), (q2, s)] + ([(q, s2)] if s2.shape != s.shape else [])
        for a, b in pairs:
            with pytest.raises(ValueError, match="x_[qs] must have"):
                w2a8.dequant_act_mx4(a, b, K)
            with pytest.raises(ValueError, match="x_[qs] must have"):
                w2a8.gemm_w4mx4(w, a, b, N, K)
            with pytest.raises(ValueError, match="x_[qs] must have"):
                w2a8.gemm_w2mx4(t, a, b, 1.0, N, K)


# ---------------------------------------------------------------------------
# launch plans
# ---------------------------------------------------------------------------
OUTPUTS = [(True, False), (False, True), (True, True)]


def test_plan_query_refuses():
    L = w2a8.lib()
    out = [ctypes.byref(ctypes.c_int()) for _ in range(5)]
    ok = (40, 100, 200, 0, 1, 256)
    assert L.w2a8_mx4_plan(*ok, *out) == 0
    for i in range(5):
        assert L.w2a8_mx4_plan(*ok, *out[:i], None, *out[i + 1:]) == NULL
    for i, bad in ((0, 0), (1, 0), (2, 0), (0, (1 << 20) + 1), (1, (1 << 30) + 1), (2, 1048449)):
        assert L.w2a8_mx4_plan(*ok[:i], bad, *ok[i + 1:], *out) == SHAPE
    for i, bad in ((4, 0), (4, 4), (5, 0), (5, 65537), (5, (1 << 31) - 1)):
        assert L.w2a8_mx4_plan(*ok[:i], bad, *ok[i + 1:], *out) == VALUE
    with pytest.raises(w2a8.W2A8Error):
        w2a8.mx4_plan(40, 100, 200, 256, f32=False)


@pytest.mark.parametrize("kind", ["w4", "w2"])
def test_test_sizes_reach_every_tile_and_store(kind):
    """The sizes that the GPU tests run take every output tile, for each
    selection of outputs, with rounds to spare, and both kinds of stores
    wherever sizes at random find them."""
    plan = lambda size, out: w2a8.mx4_plan(*size, mx4_sizes.CUS, kind == "w2", *out)
    tiles = mx4_sizes.TILES[kind]
    for i, size in enumerate(mx4_sizes.ROUNDS[kind]):
        kernel, rows, cols, groups, _ = plan(size, OUTPUTS[0])
        assert kernel == 2
        if i < len(tiles):
            assert (rows, cols, groups) == tiles[i], size
        KT = -(-size[2] // 128)
        left = KT % (4 * groups)
        assert KT >= 12 * groups and (left > 4 if groups > 1 else left % 4), size
    seen = {(plan(size, out)[1:], out) for out in OUTPUTS
            for size in mx4_sizes.ROUNDS[kind] + mx4_sizes.STAY[kind]}
    for size in mx4_sizes.STAY[kind]:
        assert all(plan(size, out)[4] == 0 for out in OUTPUTS), size
    rng = np.random.default_rng(1)
    top = np.log([60000, 60000, 27648])
    for size in np.exp(rng.uniform(0, 1, (60000, 3)) * top).round().astype(int).tolist():
        if size[0] * size[1] <= 2 ** 25:
            for out in OUTPUTS:
                p = plan(size, out)
                if p[0] == 2:
                    assert p[1:4] in tiles, size
                    assert (p[1:], out) in seen, (size, p, out)


@pytest.mark.parametrize("kind", ["w4", "w2"])
def test_test_sizes_reach_every_form_of_the_stream(kind):
    for size, (rows, waves) in zip(mx4_sizes.STREAM[kind], mx4_sizes.STREAM_FORMS, strict=True):
        p = w2a8.mx4_plan(*size, mx4_sizes.CUS, kind == "w2")
        assert p == (1, rows, 32 if kind == "w2" else 16, waves, 0), size
        assert -(-size[2] // 512) >= 3 * waves, size


# ---------------------------------------------------------------------------
# sources
# ---------------------------------------------------------------------------
@pytest.mark.skipif(shutil.which("hipcc") is None, reason="needs hipcc")
def test_kernels_claim_no_alignment_that_rows_lack():
    """Rows of results start wherever N puts them: no 16-byte access may be
    made through a pointer whose type claims 16-byte alignment."""
    csrc = os.path.join(ROOT, "w2a8_gemv_amd", "csrc")
    srcs = [os.path.join(csrc, f) for f in sorted(os.listdir(csrc)) if "mx4" in f and f.endswith(".hip")]
    assert len(srcs) == 5
    res = subprocess.run(["hipcc", "--offload-arch=gfx950", "-std=c++17", "-fsyntax-only",
                          "-Werror=align-mismatch", "-I", os.path.join(ROOT, "include"), "-I", csrc, *srcs],
                         capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]
