"""CPU tests of the operators around the ternary layers: the reference on
worked values, host packers and size queries against it, and the refusals of
every entry point (rejected before any HIP call: the stand-in pointers are
never read)."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import block_sizes
import w2a8_gemv_amd as w2a8
from conftest import ROOT
from oracle import block

NULL, SHAPE, ALIGN, VALUE, BUFSIZE = 1, 2, 3, 4, 5
FAKE = 0x10000
FAR = 0x100000000                   # stand-in buffers this far apart


# ---------------------------------------------------------------------------
# the reference itself
# ---------------------------------------------------------------------------
def test_reference_norm_of_worked_values():
    # mean(h^2) = (9 + 16) / 2; codes by the largest of 3 and 8
    q, s = block.rmsnorm_quant(np.array([[3.0, -4.0]]), np.array([1.0, 2.0]), 0.0)
    assert q.tolist() == [[48.0, -127.0]]                       # 3 * 127 / 8 = 47.6
    np.testing.assert_allclose(s, [8 / 127 / np.sqrt(12.5)], rtol=1e-15)
    q, s = block.rmsnorm_quant(np.zeros((1, 3)), None, 0.0)
    assert not q.any() and s.tolist() == [0.0]
    for bad in (np.nan, np.inf):
        q, s = block.rmsnorm_quant(np.array([[1.0, bad], [1.0, 1.0]]), None, 0.0)
        assert not q[0].any() and np.isnan(s[0]) and q[1].tolist() == [127, 127]


def test_reference_route_of_worked_values():
    inf = np.inf
    r = block.moe_route(np.array([[0, 2, 2, 1.0], [-inf, 0, -inf, -inf], [-inf] * 4, [0, inf, 0, 0],
                                  [0, 0, np.nan, 0]]), 2, True)
    assert [e for e, _ in r[0]] == [1, 2] and [p for _, p in r[0]] == [0.5, 0.5]
    assert r[1] == [(1, 1.0)] and r[2] == [] and r[3] is None and r[4] is None
    whole = block.moe_route(np.array([[0.0, 0, 0, 0]]), 3, False)[0]
    assert whole == [(0, 0.25), (1, 0.25), (2, 0.25)]


def test_reference_moe_is_a_linear_map_of_one_expert():
    """One expert whose gate is constant: y = p * w_down . quantized(u * g^2)."""
    x = np.array([[127, 0], [0, 127]], np.int8)
    eye = np.eye(2, dtype=np.int8)[None]
    one = np.ones(1, np.float32)
    y, bound = block.moe(x, np.full(2, 1 / 127, np.float32), np.zeros((2, 1)), eye, eye, eye, one, one, one, 1,
                         "relu2", True)
    np.testing.assert_allclose(y, np.eye(2), rtol=2 ** -20)
    assert not bound.any()


# ---------------------------------------------------------------------------
# sizes and packers
# ---------------------------------------------------------------------------
def w4_weights(N, K, group, zeros, seed):
    rng = np.random.default_rng(seed)
    groups = -(-K // group)
    q = rng.integers(0, 16, (N, K)).astype(np.uint8)
    scales = torch.from_numpy(rng.uniform(0.5, 2, (N, groups)).astype(np.float32))
    z = rng.integers(0, 16, (N, groups)).astype(np.uint8) if zeros else None
    return q, scales, z


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,K", [(1, 1), (3, 33), (16, 128), (17, 127), (33, 300), (5, 1000)])
def test_w4_packers_match_the_reference(N, K, group, zeros, dtype):
    q, scales, z = w4_weights(N, K, group, zeros, N * K + group)
    scales = scales.to(dtype)
    inter = torch.from_numpy(block.w4_interchange(q))
    zt = None if z is None else torch.from_numpy(z)
    packed = w2a8.pack_w4a8(inter, scales, N, K, group, zt)
    want = block.w4_packed(q, scales.view(torch.int16).numpy().view(np.uint16), z, group)
    assert packed.numel() == want.size == w2a8.w4a8_packed_bytes(N, K, group, zeros)
    np.testing.assert_array_equal(packed.numpy(), want)
    c, s, zz = w2a8.unpack_w4a8(packed, N, K, group, dtype, zeros)
    np.testing.assert_array_equal(c.numpy(), inter.numpy())
    assert torch.equal(s.view(torch.int16), scales.view(torch.int16))
    assert (zz is None) == (z is None) and (z is None or np.array_equal(zz.numpy(), z))


def test_w4_packers_refuse():
    L = w2a8.lib()
    N, K, g = 4, 40, 32
    c, s, z = np.zeros((4, 20), np.uint8), np.zeros((4, 2), np.uint16), np.zeros((4, 2), np.uint8)
    out = np.zeros(w2a8.w4a8_packed_bytes(N, K, g, True), np.uint8)
    cp, sp, zp, op, n = c.ctypes.data, s.ctypes.data, z.ctypes.data, out.ctypes.data, out.size
    p = lambda c=cp, s=sp, z=zp, N=N, K=K, g=g, o=op, n=n: L.pack_w4a8(c, s, z, N, K, g, o, n)
    u = lambda o=op, n=n, N=N, K=K, g=g, c=cp, s=sp, z=zp: L.unpack_w4a8(o, n, N, K, g, c, s, z)
    for f in (p, u):
        assert f() == 0 and f(z=None) == 0
        assert f(c=None) == NULL and f(s=None) == NULL and f(o=None) == NULL
        assert f(N=0) == SHAPE and f(K=0) == SHAPE and f(K=1048449) == SHAPE
        assert f(g=16) == VALUE and f(g=0) == VALUE and f(g=256) == VALUE and f(n=n - 1) == BUFSIZE
    z[3, 1] = 16
    assert p() == VALUE
    for bad in ((0, 5, 32), (5, 0, 32), (5, 5, 33), ((1 << 30) + 1, 5, 32), (5, 1048449, 128)):
        assert L.w4a8_packed_bytes(*bad, 0) == -1
        with pytest.raises(w2a8.W2A8Error):
            w2a8.w4a8_packed_bytes(*bad)
    assert L.w4a8_packed_bytes(1 << 30, 1048448, 32, 1) > 0
    t = torch.zeros
    with pytest.raises(ValueError):
        w2a8.pack_w4a8(t((4, 19), dtype=torch.uint8), t((4, 2), dtype=torch.float16), 4, 40, 32)
    with pytest.raises(ValueError):
        w2a8.pack_w4a8(t((4, 20), dtype=torch.uint8), t((4, 1), dtype=torch.float16), 4, 40, 32)
    with pytest.raises(TypeError):
        w2a8.pack_w4a8(t((4, 20), dtype=torch.uint8), t((4, 2)), 4, 40, 32)
    with pytest.raises(w2a8.W2A8Error):
        w2a8.unpack_w4a8(t(n - 1, dtype=torch.uint8), 4, 40, 32, zeros=True)


def test_moe_workspace_query():
    L = w2a8.lib()
    ok = (64, 5120, 6912, 256, 16)
    assert L.w2a8_moe_workspace_bytes(*ok) >= 4 * 64 * 16 * (5120 + 6912)
    for i, bad in ((0, 0), (0, 65), (1, 0), (1, 1048449), (2, 0), (2, 1048449), (3, 0), (3, 257), (4, 0), (4, 17)):
        assert L.w2a8_moe_workspace_bytes(*ok[:i], bad, *ok[i + 1:]) == -1
    assert L.w2a8_moe_workspace_bytes(1, 1, 1, 3, 4) == -1
    with pytest.raises(w2a8.W2A8Error):
        w2a8.w2a8_moe_workspace_bytes(1, 1, 1, 3, 4)


# ---------------------------------------------------------------------------
# refusals of the device entry points
# ---------------------------------------------------------------------------
def apart(names):
    return {n: FAR * (i + 1) for i, n in enumerate(names)}


def norm_call(**kw):
    a = dict(apart(["x", "r", "w", "h", "q", "s"]), t=1, M=3, K=40, eps=1e-5)
    a.update(kw)
    return w2a8.lib().rmsnorm_quant_int8(a["x"], a["r"], a["w"], a["t"], a["M"], a["K"], a["eps"], a["h"], a["q"],
                                         a["s"], None)


def w4_call(**kw):
    a = dict(apart(["w", "x", "s", "f", "b", "ws"]), M=3, N=40, K=200, g=64, t=2, z=1, n=0)
    a.update(kw)
    return w2a8.lib().w4a8_gemm(a["w"], a["x"], a["s"], a["M"], a["N"], a["K"], a["g"], a["t"], a["z"], a["f"],
                                a["b"], a["ws"], a["n"], None)


MOE_IN = {"x": 3 * 200, "sa": 12, "l": 3 * 6 * 2, "wg": 0, "wu": 0, "wd": 0, "sg": 24, "su": 24, "sd": 24}


def moe_call(**kw):
    names = list(MOE_IN) + ["f", "b", "ws"]
    a = dict(apart(names), t=1, M=3, H=200, I=100, E=6, k=2, act=0, re=1)
    a["n"] = w2a8.w2a8_moe_workspace_bytes(3, 200, 100, 6, 2)
    a.update(kw)
    return w2a8.lib().w2a8_moe(a["x"], a["sa"], a["l"], a["t"], a["wg"], a["wu"], a["wd"], a["sg"], a["su"], a["sd"],
                               a["M"], a["H"], a["I"], a["E"], a["k"], a["act"], a["re"], a["f"], a["b"], a["ws"],
                               a["n"], None)


def test_norm_refuses():
    for name in ("x", "q", "s", "h"):
        assert norm_call(**{name: None}) == NULL
    assert norm_call(r=None) == VALUE                       # h without a residual
    assert norm_call(M=0) == SHAPE and norm_call(M=(1 << 20) + 1) == SHAPE
    assert norm_call(K=0) == SHAPE and norm_call(K=1048449) == SHAPE
    assert norm_call(t=-1) == VALUE and norm_call(t=3) == VALUE
    for eps in (-1e-9, float("nan"), float("inf")):
        assert norm_call(eps=eps) == VALUE
    for name in "xrwhq":
        assert norm_call(**{name: FAKE + 8}) == ALIGN
    assert norm_call(s=FAKE + 2) == ALIGN
    at, n = apart(["x", "r", "w", "h", "q", "s"]), {"x": 240, "r": 240, "w": 80, "h": 240, "q": 120, "s": 12}
    for out in "hqs":
        for other in "xrwhqs":
            if out == other:
                continue
            assert norm_call(**{out: at[other] + (n[other] - 1) // 16 * 16}) == VALUE
            assert norm_call(**{other: at[out] + (n[out] - 1) // 16 * 16}) == VALUE
    assert norm_call(h=at["x"] + 16) == VALUE               # in place, but moved


def test_w4_gemm_refuses():
    for name in ("w", "x", "s"):
        assert w4_call(**{name: None}) == NULL
    assert w4_call(f=None, b=None) == NULL
    assert w4_call(M=0) == SHAPE and w4_call(M=65) == SHAPE
    assert w4_call(N=0) == SHAPE and w4_call(N=(1 << 30) + 1) == SHAPE and w4_call(K=0) == SHAPE
    assert w4_call(K=1048449) == SHAPE
    assert w4_call(g=16) == VALUE and w4_call(g=256) == VALUE and w4_call(t=0) == VALUE and w4_call(t=3) == VALUE
    for name in "wxfb":
        assert w4_call(**{name: FAKE + 8}) == ALIGN
    assert w4_call(s=FAKE + 2) == ALIGN
    at = apart(["w", "x", "s", "f", "b"])
    n = {"w": w2a8.w4a8_packed_bytes(40, 200, 64, True), "x": 600, "s": 12, "f": 480, "b": 240}
    for out in "fb":
        for other in "wxsfb":
            if out != other:
                assert w4_call(**{out: at[other] + (n[other] - 1) // 16 * 16}) == VALUE
                assert w4_call(**{other: at[out] + (n[out] - 1) // 16 * 16}) == VALUE


def test_w4_gemm_refuses_workspaces():
    L = w2a8.lib()
    assert L.w4a8_workspace_bytes(1, 1 << 30, 1048448) == 0 and L.w4a8_workspace_bytes(64, 40, 2047 - 128) == 0
    for bad in ((0, 5, 5), (65, 5, 5), (5, 0, 5), (5, (1 << 30) + 1, 5), (5, 5, 0), (5, 5, 1048449)):
        assert L.w4a8_workspace_bytes(*bad) == -1
        with pytest.raises(w2a8.W2A8Error):
            w2a8.w4a8_workspace_bytes(*bad)
    big = dict(M=3, N=40, K=6400)
    need = w2a8.w4a8_workspace_bytes(3, 40, 6400)
    assert need == 4 * 3 * 40 * 6
    assert w4_call(**big, ws=None, n=need) == NULL and w4_call(**big, n=need - 1) == BUFSIZE
    assert w4_call(**big, ws=FAKE + 8, n=need) == ALIGN
    at = apart(["w", "x", "s", "f", "b", "ws"])
    n = {"w": w2a8.w4a8_packed_bytes(40, 6400, 64, True), "x": 3 * 6400, "s": 12, "f": 480, "b": 240, "ws": need}
    for other in "wxsfb":
        assert w4_call(**big, n=need, **{"ws": at[other] + (n[other] - 1) // 16 * 16}) == VALUE
        assert w4_call(**big, n=need, **{other: at["ws"] + (need - 1) // 16 * 16}) == VALUE


def test_moe_refuses():
    for name in list(MOE_IN) + ["ws"]:
        assert moe_call(**{name: None}) == NULL, name
    assert moe_call(f=None, b=None) == NULL
    for name, bad in (("M", 0), ("M", 65), ("H", 0), ("H", 1048449), ("I", 0), ("I", 1048449), ("E", 0), ("E", 257),
                      ("k", 0), ("k", 7)):
        assert moe_call(**{name: bad}) == SHAPE, (name, bad)
    assert moe_call(E=30, k=17) == SHAPE
    assert moe_call(t=-1) == VALUE and moe_call(t=3) == VALUE and moe_call(act=2) == VALUE and moe_call(act=-1) == VALUE
    for name in ("x", "l", "wg", "wu", "wd", "f", "b", "ws"):
        assert moe_call(**{name: FAKE + 8}) == ALIGN, name
    for name in ("sa", "sg", "su", "sd"):
        assert moe_call(**{name: FAKE + 2}) == ALIGN, name
    need = w2a8.w2a8_moe_workspace_bytes(3, 200, 100, 6, 2)
    assert moe_call(n=need - 1) == BUFSIZE
    n = dict(MOE_IN, wg=6 * w2a8.packed_bytes(100, 200), wu=6 * w2a8.packed_bytes(100, 200),
             wd=6 * w2a8.packed_bytes(200, 100), f=2400, b=1200, ws=need)
    at = apart(n)
    for out in ("f", "b", "ws"):
        for other in n:
            if out != other:
                assert moe_call(**{out: at[other] + (n[other] - 1) // 16 * 16}) == VALUE, (out, other)
                assert moe_call(**{other: at[out] + (n[out] - 1) // 16 * 16}) == VALUE, (out, other)


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    x8, s, u8 = torch.zeros((2, 64), dtype=torch.int8), torch.zeros(2), torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(ValueError):
        w2a8.rmsnorm_quant_int8(x)
    with pytest.raises(TypeError):
        w2a8.rmsnorm_quant_int8(x.double())
    with pytest.raises(TypeError):
        w2a8.rmsnorm_quant_int8([1.0])
    with pytest.raises(ValueError):
        w2a8.gemm_w4a8(u8, x8, s, 16, 64, 32)
    with pytest.raises(ValueError):
        w2a8.linear_w4a8(x, u8, 16, 64, 32)
    with pytest.raises(ValueError):
        w2a8.moe(x8, s, torch.zeros(2, 3), u8, u8, u8, s, s, s, 64, 64, 1)


@pytest.fixture
def host_as_gpu(monkeypatch):
    """The binding's checks on host tensors, with the library's calls in a list instead."""
    calls = []

    class Lib:
        def __getattr__(self, name):
            real = getattr(library, name)
            if name in ("rmsnorm_quant_int8", "w4a8_gemm", "w2a8_moe"):
                return lambda *a: calls.append((name, a)) or 0
            return real
    library = w2a8.lib()
    monkeypatch.setattr(w2a8, "_mx4_gpu", lambda t, name: t.get_device())
    monkeypatch.setattr(w2a8, "_mx4_stream", lambda stream, index: None)
    monkeypatch.setattr(w2a8, "lib", lambda: Lib())
    return calls


def test_binding_checks_of_the_norm(host_as_gpu):
    t = torch.zeros
    x, w = t(3, 40, dtype=torch.bfloat16), t(40, dtype=torch.bfloat16)
    q, s, h = w2a8.rmsnorm_quant_int8(x, w)
    assert q.shape == (3, 40) and s.shape == (3,) and h is x
    q, s, h = w2a8.rmsnorm_quant_int8(x[0], w, residual=x[1])
    assert q.shape == (1, 40) and h.shape == (40,) and h.dtype == x.dtype
    assert w2a8.rmsnorm_quant_int8(x, residual=w.expand(3, 40).contiguous(), h=x)[2] is x
    for kw, err in (({"weight": w[:39]}, ValueError), ({"weight": w.float()}, TypeError), ({"residual": x[:2]}, ValueError),
                    ({"residual": x.float()}, TypeError), ({"h": x}, ValueError),
                    ({"residual": x, "h": x[:2]}, ValueError), ({"x_q": t(3, 39, dtype=torch.int8)}, ValueError),
                    ({"s_a": t(2)}, ValueError), ({"s_a": t(3).double()}, TypeError)):
        with pytest.raises(err):
            w2a8.rmsnorm_quant_int8(x, **kw)
    with pytest.raises(ValueError):
        w2a8.rmsnorm_quant_int8(t(40, 3, dtype=torch.bfloat16).t())
    with pytest.raises(ValueError):
        w2a8.rmsnorm_quant_int8(t(2, 3, 4))


def test_binding_checks_of_the_products(host_as_gpu):
    t = torch.zeros
    x, s = t((3, 40), dtype=torch.int8), t(3)
    w = t(w2a8.w4a8_packed_bytes(20, 40, 32, True), dtype=torch.uint8)
    assert w2a8.gemm_w4a8(w, x, s, 20, 40, 32, zeros=True).shape == (3, 20)
    y = w2a8.gemm_w4a8(w, x[0], s[:1], 20, 40, 32, torch.bfloat16, True, torch.bfloat16)
    assert y.shape == (1, 20) and y.dtype == torch.bfloat16
    assert host_as_gpu[-1][1][7:9] == (1, 1) and host_as_gpu[-2][1][7:9] == (2, 1)
    long = t((3, 6400), dtype=torch.int8)
    wl = t(w2a8.w4a8_packed_bytes(20, 6400, 32), dtype=torch.uint8)
    w2a8.gemm_w4a8(wl, long, s, 20, 6400, 32)
    need = w2a8.w4a8_workspace_bytes(3, 20, 6400)
    assert need > 0 and host_as_gpu[-1][1][-2] == need
    y = t(3, 20)
    w2a8.w4a8_gemm(wl, long, s, 3, 20, 6400, 32, y_f32=y, workspace=t(need, dtype=torch.uint8))
    with pytest.raises(ValueError):
        w2a8.w4a8_gemm(wl, long, s, 3, 20, 6400, 32, y_f32=y, workspace=t(need - 1, dtype=torch.uint8))
    for args, kw, err in (((w[:-1], x, s, 20, 40, 32), {"zeros": True}, ValueError), ((w, x, s, 20, 39, 32), {}, ValueError),
                          ((w, x, s[:2], 20, 40, 32), {}, ValueError), ((w, x.short(), s, 20, 40, 32), {}, TypeError),
                          ((w, x, s, 20, 40, 48), {}, w2a8.W2A8Error),
                          ((w, x, s, 20, 40, 32), {"scale_dtype": torch.float32}, TypeError),
                          ((w, x, s, 20, 40, 32), {"out_dtype": torch.float16}, TypeError)):
        with pytest.raises(err):
            w2a8.gemm_w4a8(*args, **kw)


def test_binding_refuses_weights_of_another_form(host_as_gpu):
    t = torch.zeros
    x, s = t((3, 300), dtype=torch.int8), t(3)
    for group in (32, 64, 128):
        for zeros in (False, True):
            w = t(w2a8.w4a8_packed_bytes(20, 300, group, zeros), dtype=torch.uint8)
            w2a8.gemm_w4a8(w, x, s, 20, 300, group, zeros=zeros)
            with pytest.raises(ValueError):
                w2a8.gemm_w4a8(w, x, s, 20, 300, group, zeros=not zeros)
            with pytest.raises(ValueError):
                w2a8.gemm_w4a8(torch.cat([w, w[:16]]), x, s, 20, 300, group, zeros=zeros)


def test_workspace_of_the_products():
    """None for one row and for short rows; room for the parts that are planned everywhere."""
    for K in (1, 1919, 1920):
        assert w2a8.w4a8_workspace_bytes(64, 100, K) == 0
    assert w2a8.w4a8_workspace_bytes(1, 100, 50000) == 0
    for M in (2, 16, 17, 33, 64):
        for N in (1, 17, 640, 5120, 9000):
            for K in (100, 1920, 1921, 2049, 5120, 50000):
                for group in (32, 64, 128):
                    parts = w2a8.w4a8_plan(M, N, K, group, 256)[3]
                    assert parts == 1 or 4 * M * N * parts <= w2a8.w4a8_workspace_bytes(M, N, K)


def test_binding_checks_of_the_mixture(host_as_gpu):
    t, u8 = torch.zeros, torch.uint8
    H, I, E = 40, 33, 5
    a = dict(x_q=t((3, H), dtype=torch.int8), s_a=t(3), logits=t(3, E), w_gate=t((E, w2a8.packed_bytes(I, H)), dtype=u8),
             w_up=t((E, w2a8.packed_bytes(I, H)), dtype=u8), w_down=t((E, w2a8.packed_bytes(H, I)), dtype=u8),
             s_gate=t(E), s_up=t(E), s_down=t(E), H=H, I=I, top_k=2)
    assert w2a8.moe(**a).shape == (3, H)
    one = dict(a, x_q=a["x_q"][0], s_a=a["s_a"][:1], logits=a["logits"][0])
    assert w2a8.moe(**one, out_dtype=torch.bfloat16).shape == (1, H)
    for kw, err in (({"H": 41}, ValueError), ({"I": 70}, ValueError), ({"top_k": 6}, w2a8.W2A8Error),
                    ({"logits": t(2, E)}, ValueError), ({"logits": t(3, E).double()}, TypeError), ({"logits": None}, TypeError),
                    ({"s_up": t(E - 1)}, ValueError), ({"w_gate": a["w_gate"][1:]}, ValueError),
                    ({"w_down": a["w_down"].int()}, TypeError), ({"activation": "gelu"}, ValueError),
                    ({"s_a": t(4)}, ValueError), ({"out_dtype": torch.float16}, TypeError),
                    ({"s_gate": [1.0] * E}, TypeError), ({"w_up": a["w_up"].t()}, ValueError)):
        with pytest.raises(err):
            w2a8.moe(**{**a, **kw})
    y = t(3, H)
    raw = [a[n] for n in ("x_q", "s_a", "logits", "w_gate", "w_up", "w_down", "s_gate", "s_up", "s_down")]
    need = w2a8.w2a8_moe_workspace_bytes(3, H, I, E, 2)
    w2a8.w2a8_moe(*raw, 3, H, I, E, 2, y_f32=y, workspace=t(need, dtype=u8))
    assert host_as_gpu[-1][1][-2] == need
    with pytest.raises(ValueError):
        w2a8.w2a8_moe(*raw, 3, H, I, E, 2, y_f32=y, workspace=t(need - 1, dtype=u8))


# ---------------------------------------------------------------------------
# launch plans
# ---------------------------------------------------------------------------
def test_plan_queries_refuse():
    L = w2a8.lib()
    out = [ctypes.byref(ctypes.c_int()) for _ in range(4)]
    for f, ok, n in ((L.w2a8_w4a8_plan, (40, 100, 200, 64, 256), 4), (L.w2a8_moe_plan, (40, 100, 200, 8, 2, 256), 3)):
        assert f(*ok, *out[:n]) == 0
        for i in range(n):
            assert f(*ok, *out[:i], None, *out[i + 1:n]) == NULL
        for i in range(len(ok) - 1):
            assert f(*ok[:i], 0, *ok[i + 1:], *out[:n]) == (VALUE if n == 4 and i == 3 else SHAPE)
        for bad in (0, 65537, (1 << 31) - 1):
            assert f(*ok[:-1], bad, *out[:n]) == VALUE
    assert L.w2a8_w4a8_plan(65, 100, 200, 64, 256, *out) == SHAPE
    assert L.w2a8_w4a8_plan(40, 100, 200, 48, 256, *out) == VALUE
    assert L.w2a8_moe_plan(65, 100, 200, 8, 2, 256, *out[:3]) == SHAPE
    assert L.w2a8_tune_moe(-1) == VALUE and L.w2a8_tune_moe(5) == VALUE and L.w2a8_tune_moe(0) == 0


def test_test_sizes_reach_every_plan():
    for want, sizes in block_sizes.W4.items():
        for size in sizes:
            for group in (32, 64, 128):
                p = w2a8.w4a8_plan(*size, group, block_sizes.CUS)
                assert p[:3] + (p[3] > 1,) == want, (size, group, p)
    for want, sizes in block_sizes.MOE.items():
        for size in sizes:
            assert w2a8.moe_plan(*size, block_sizes.CUS) == want, size
    rng = np.random.default_rng(1)
    for m, n, k in np.exp(rng.uniform(0, 1, (20000, 3)) * np.log([64, 200000, 100000])).round().astype(int).tolist():
        p = w2a8.w4a8_plan(m, n, k, 32 << (m + n + k) % 3, block_sizes.CUS)
        waves = p[2] if p[0] != 2 else 0
        assert p[:3] + (p[3] > 1,) in block_sizes.W4 or (waves and waves == min(-(-k // 128), 4 if p[0] == 1 and n > 8192 else 8)), (m, n, k, p)
        assert p[3] == 1 or 4 * m * n * p[3] <= w2a8.w4a8_workspace_bytes(m, n, k)


def test_moe_knob():
    sizes = (8, 1300, 4001, 6, 3)
    try:
        want = {0: w2a8.moe_plan(*sizes, 256), 1: (1, 1, 1), 3: (2, 1, 1), 4: (2, 2, 2)}
        assert want[0][0] == 2
        for mode, plan in want.items():
            w2a8.tune_moe(mode)
            assert w2a8.moe_plan(*sizes, 256) == plan
        w2a8.tune_moe(1)
        assert w2a8.moe_plan(1, 40, 50000, 3, 1, 256)[0] == 2          # does not fit LDS
        w2a8.tune_moe(2)
        assert w2a8.moe_plan(1, 40, 40, 3, 1, 256)[0] == 2
    finally:
        w2a8.tune_moe(0)


# ---------------------------------------------------------------------------
# sources
# ---------------------------------------------------------------------------
@pytest.mark.skipif(shutil.which("hipcc") is None, reason="needs hipcc")
def test_kernels_claim_no_alignment_that_rows_lack():
    """Rows start wherever their length puts them: no access may be made through a pointer whose
    type claims more alignment than its elements have."""
    csrc = os.path.join(ROOT, "w2a8_gemv_amd", "csrc")
    srcs = [os.path.join(csrc, f) for f in ("rmsnorm.hip", "w4a8.hip", "moe.hip", "host_block.hip")]
    res = subprocess.run(["hipcc", "--offload-arch=gfx950", "-std=c++17", "-fsyntax-only",
                          "-Werror=align-mismatch", "-I", os.path.join(ROOT, "include"), "-I", csrc, *srcs],
                         capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]
