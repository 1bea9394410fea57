"""Argument checks of the 4-bit weight calls and pins of their 64-bit oracle (no GPU).

Pointers are fake, never-dereferenced addresses: every call here must be refused on the host."""
import os

import numpy as np
import pytest
import torch

from oracle import w4 as ref
from w4_util import gen_w4

A = 0x10000


@pytest.fixture(scope="module")
def q():
    from skinny_gemm_qlin_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from skinny_gemm_qlin_amd import _build
        _build.build()
    return _lib.load()


SHAPES = [({"M": 0}, -2), ({"M": 16385}, -2), ({"N": 0}, -2), ({"N": (1 << 20) + 2}, -2), ({"K": 0}, -2),
          ({"K": 48, "ldw": 64, "group": 16}, -2), ({"K": (1 << 20) + 32}, -2), ({"group": 0}, -2),
          ({"group": 16}, -2), ({"group": 96}, -2), ({"group": -32}, -2), ({"group": 2048}, -2),
          ({"dtype": 2}, -6), ({"dtype": -1}, -6), ({"w": None}, -1), ({"ws": None}, -1),
          ({"ldw": 496}, -3), ({"ldw": (1 << 20) + 16}, -3), ({"ldw": 520}, -4), ({"w": A + 8}, -4), ({"ws": A + 1}, -4)]


def _with(defaults, changes):
    d = dict(defaults)
    d.update(changes)
    return d


@pytest.mark.parametrize("change,status", SHAPES + [
    ({"x": None}, -1), ({"y": None}, -1), ({"ldx": 1016}, -3), ({"ldy": 63}, -3), ({"x": A + 2}, -4),
    ({"ldx": 1028}, -4), ({"y": A + 1}, -4), ({"bias": A + 1}, -4)])
def test_gemv_w4_refusals(q, change, status):
    a = _with(dict(x=A, ldx=1024, M=1, K=1024, dtype=0, w=A, ldw=512, N=64, ws=A, wz=None, group=128, bias=None, y=A,
                   ldy=64), change)
    if "K" in change and "ldx" not in change:
        a["ldx"] = 1 << 21
        a["ldw"] = 1 << 20
    if "N" in change:
        a["ldy"] = 1 << 21
    assert q.qlin_gemv_w4(a["x"], a["ldx"], a["M"], a["K"], a["dtype"], a["w"], a["ldw"], a["N"], a["ws"], a["wz"],
                          a["group"], a["bias"], a["y"], a["ldy"], None) == status


@pytest.mark.parametrize("change,status", SHAPES + [
    ({"dy": None}, -1), ({"dx": None}, -1), ({"lddy": 56}, -3), ({"lddx": 1023}, -3), ({"dy": A + 2}, -4),
    ({"lddy": 68}, -4), ({"dx": A + 1}, -4), ({"work": None, "N": 65536}, -5), ({"size": 16, "N": 65536}, -5),
    ({"work": A + 4, "N": 65536}, -4)])
def test_gemv_w4_bwd_refusals(q, change, status):
    a = _with(dict(dy=A, lddy=64, M=1, N=64, dtype=0, w=A, ldw=512, K=1024, ws=A, wz=A, group=128, dx=A, lddx=1024,
                   work=A, size=1 << 40), change)
    if "N" in change:
        a["lddy"] = 1 << 21
    if "K" in change:
        a["lddx"] = 1 << 21
        a["ldw"] = 1 << 20
    assert q.qlin_gemv_w4_bwd(a["dy"], a["lddy"], a["M"], a["N"], a["dtype"], a["w"], a["ldw"], a["K"], a["ws"],
                              a["wz"], a["group"], a["dx"], a["lddx"], a["work"], a["size"], None) == status


def test_bwd_workspace(q):
    f = q.qlin_gemv_w4_bwd_workspace_bytes
    assert f(0, 64, 64) == 0 and f(1, 64, 40) == 0 and f(1, 0, 64) == 0 and f(20000, 64, 64) == 0
    b = f(1, 65536, 1024)
    assert b > 0 and b % (4 * 1024) == 0


@pytest.mark.parametrize("change,status", SHAPES + [
    ({"act": 2}, -6), ({"act": -1}, -6), ({"x": None}, -1), ({"y": None}, -1), ({"ldx": 1016}, -3),
    ({"ldy": 31}, -3), ({"gu": A, "ldgu": 63}, -3), ({"gu": A + 1}, -4), ({"x": A + 8}, -4), ({"y": A + 1}, -4)])
def test_glu_w4_refusals(q, change, status):
    a = _with(dict(x=A, ldx=1024, M=1, K=1024, dtype=1, w=A, ldw=512, N=64, ws=A, wz=None, group=128, act=0, y=A,
                   ldy=64, gu=None, ldgu=64), change)
    if "K" in change:
        a["ldx"] = 1 << 21
        a["ldw"] = 1 << 20
    if "N" in change:
        a["ldy"] = a["ldgu"] = 1 << 22
    assert q.qlin_glu_w4(a["x"], a["ldx"], a["M"], a["K"], a["dtype"], a["w"], a["ldw"], a["N"] // 2, a["ws"],
                         a["wz"], a["group"], a["act"], a["y"], a["ldy"], a["gu"], a["ldgu"], None) == status


@pytest.mark.parametrize("change,status", SHAPES + [
    ({"act": 7}, -6), ({"x": None, "gu": None}, -1), ({"dy": None}, -1), ({"dgu": None}, -1), ({"lddy": 31}, -3),
    ({"gu": A, "ldgu": 63}, -3), ({"gu": None, "ldx": 1016}, -3), ({"lddgu": 56}, -3), ({"lddx": 1016}, -3),
    ({"dy": A + 1}, -4), ({"gu": A + 1}, -4), ({"gu": None, "x": A + 2}, -4), ({"dgu": A + 8}, -4),
    ({"lddgu": 68}, -4), ({"dx": A + 1}, -4), ({"work": None, "N": 65536}, -5), ({"size": 8, "N": 65536}, -5)])
def test_glu_w4_bwd_refusals(q, change, status):
    a = _with(dict(dy=A, lddy=64, M=1, N=64, dtype=0, act=0, x=A, ldx=1024, gu=A, ldgu=64, w=A, ldw=512, K=1024, ws=A,
                   wz=A, group=128, dgu=A, lddgu=64, dx=A, lddx=1024, work=A, size=1 << 40), change)
    if "K" in change:
        a["ldx"] = a["lddx"] = 1 << 21
        a["ldw"] = 1 << 20
    if "N" in change:
        a["lddy"] = a["ldgu"] = a["lddgu"] = 1 << 22
    assert q.qlin_glu_w4_bwd(a["dy"], a["lddy"], a["M"], a["N"] // 2, a["dtype"], a["act"], a["x"], a["ldx"], a["gu"],
                             a["ldgu"], a["w"], a["ldw"], a["K"], a["ws"], a["wz"], a["group"], a["dgu"], a["lddgu"],
                             a["dx"], a["lddx"], a["work"], a["size"], None) == status


# ----------------------------------------------------------------------------- the 64-bit forms themselves

def test_dense_by_hand():
    """Two rows, two groups of 32, written out: nibble order, group and zero indices."""
    w = np.zeros((2, 32), np.uint8)
    w[0, 0] = 0x3F    # elements 0, 1 = 15, 3
    w[1, 16] = 0x08   # elements 32, 33 = 8, 0
    ws = np.array([[0.5, 2.0], [4.0, 0.25]])
    W = ref.dense(w, ws, None, 32)
    assert W[0, 0] == 0.5 * 7 and W[0, 1] == 0.5 * -5 and W[0, 2] == 0.5 * -8 and W[0, 32] == 2.0 * -8
    assert W[1, 32] == 0.0 and W[1, 33] == 0.25 * -8
    wz = np.array([[1, 15], [0, 3]], np.uint8)
    W = ref.dense(w, ws, wz, 32)
    assert W[0, 0] == 0.5 * 14 and W[0, 1] == 0.5 * 2 and W[0, 40] == 2.0 * -15
    assert W[1, 0] == 0.0 and W[1, 32] == 0.25 * 5 and W[1, 33] == 0.25 * -3


@pytest.mark.parametrize("kind", [0, 1])
def test_activation_against_torch_and_differences(kind):
    g = np.linspace(-12, 12, 4001)
    a, da = ref.act(g, kind)
    t = torch.from_numpy(g)
    want = torch.nn.functional.silu(t) if kind == 0 else torch.nn.functional.gelu(t, approximate="tanh")
    assert np.allclose(a, want.numpy(), rtol=1e-13, atol=1e-15)
    h = 1e-5
    num = (ref.act(g + h, kind)[0] - ref.act(g - h, kind)[0]) / (2 * h)
    assert np.allclose(da, num, rtol=0, atol=1e-9)
    num2 = (ref.act(g + h, kind)[1] - ref.act(g - h, kind)[1]) / (2 * h)
    assert np.abs(da).max() <= ref.ACT_D1 and np.abs(num2).max() <= ref.ACT_D2


@pytest.mark.parametrize("kind", [0, 1])
def test_gradient_formula_against_differences(kind):
    """dx and dgu of the gated block against central differences of its forward form."""
    M, I, K, G = 3, 5, 64, 32
    w, ws, wz = gen_w4(2 * I, K, G, "bf16", True, seed=3)
    W = ref.dense(w, ws.float().numpy().astype(np.float64), wz, G)
    rng = np.random.default_rng(0)
    x, dy = rng.standard_normal((M, K)), rng.standard_normal((M, I))

    def loss(gu):
        return float((ref.act(gu[:, :I], kind)[0] * gu[:, I:] * dy).sum())

    gu = x @ W.T
    a, da = ref.act(gu[:, :I], kind)
    dgu = np.concatenate([dy * gu[:, I:] * da, dy * a], axis=1)
    h = 1e-6
    for m, j in [(0, 0), (1, 4), (2, 5), (0, 9)]:
        e = np.zeros_like(gu)
        e[m, j] = h
        assert abs((loss(gu + e) - loss(gu - e)) / (2 * h) - dgu[m, j]) < 1e-6 * (1 + abs(dgu[m, j]))
    dx = dgu @ W
    for m, k in [(0, 0), (1, 33), (2, 63)]:
        e = np.zeros_like(x)
        e[m, k] = h
        num = (loss((x + e) @ W.T) - loss((x - e) @ W.T)) / (2 * h)
        assert abs(num - dx[m, k]) < 1e-5 * (1 + abs(dx[m, k]))


# ----------------------------------------------------------------------------- the binding's own refusals (before any launch)

def test_binding_refusals():
    import skinny_gemm_qlin_amd as ql
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    w = torch.zeros((8, 32), dtype=torch.uint8)
    ws = torch.zeros((8, 2), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        ql.qlin_gemv_w4(x, w, ws)                                    # host tensors
    for bad in (x.float(), x.to(torch.int16)):
        with pytest.raises(TypeError):
            ql.qlin_gemv_w4(bad, w, ws)
    for name, args in [("w", (x, w.to(torch.int8), ws)), ("ws", (x, w, ws.half()))]:
        with pytest.raises((TypeError, ValueError)):
            ql.qlin_gemv_w4(*args)
        with pytest.raises((TypeError, ValueError)):
            ql.qlin_glu_w4(*args)
        with pytest.raises((TypeError, ValueError)):
            ql.qlin_gemv_w4_bwd(*args)
        with pytest.raises((TypeError, ValueError)):
            ql.qlin_glu_w4_bwd(*args, gu=args[0])


def test_fake_shapes():
    from torch._subclasses.fake_tensor import FakeTensorMode
    import skinny_gemm_qlin_amd.torch_ops  # noqa: F401
    with FakeTensorMode():
        x = torch.empty((5, 64), dtype=torch.float16)
        w, s, z = torch.empty((10, 32), dtype=torch.uint8), torch.empty((10, 2), dtype=torch.float16), None
        assert torch.ops.qlin.gemv_w4(x, w, s, z).shape == (5, 10)
        y, gu = torch.ops.qlin.glu_w4(x, w, s, z, 1, True)
        assert y.shape == (5, 5) and gu.shape == (5, 10) and gu.stride() == (16, 1) and y.dtype == torch.float16
        assert torch.ops.qlin.glu_w4(x, w, s, z)[1].shape == (0, 0)
        assert torch.ops.qlin.gemv_w4_bwd(gu, w, s, z).shape == (5, 64)
        dx, dgu = torch.ops.qlin.glu_w4_bwd(y, w, s, z, x, None, 0)
        assert dx.shape == (5, 64) and dgu.shape == (5, 10)
