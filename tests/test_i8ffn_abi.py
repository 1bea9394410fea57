"""Argument checks of the INT8 feed-forward calls, and pins of their 64-bit definition (no GPU).

Pointers are fake, never-dereferenced addresses: every call here must be refused on the host."""
import os

import numpy as np
import pytest

from oracle import i8ffn

A = 0x10000


@pytest.fixture(scope="module")
def q():
    from skinny_gemm_qlin_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from skinny_gemm_qlin_amd import _build
        _build.build()
    return _lib.load()


GLU = dict(x=A, ldx=1024, M=1, K=1024, dtype=0, w13=A, ldw=1024, I=64, s13=A, per_row=1, act=0, xq=A, ldxq=1024, xs=A, y=A,
           ldy=64)


@pytest.mark.parametrize("change,status", [
    ({"dtype": 2}, -6), ({"dtype": -1}, -6), ({"act": 2}, -6), ({"act": -1}, -6), ({"per_row": 2}, -6), ({"per_row": -1}, -6),
    ({"x": None}, -1), ({"w13": None}, -1), ({"s13": None}, -1), ({"xq": None}, -1), ({"xs": None}, -1), ({"y": None}, -1),
    ({"M": 0}, -2), ({"M": -1}, -2), ({"M": 16385}, -2), ({"I": 0}, -2), ({"I": (1 << 20) + 1, "ldy": 1 << 21}, -2),
    ({"K": 0}, -2), ({"K": 1000}, -2), ({"K": -16}, -2), ({"K": 131088, "ldx": 1 << 20, "ldw": 1 << 20, "ldxq": 1 << 20}, -2),
    ({"ldx": 1016}, -3), ({"ldw": 1008}, -3), ({"ldxq": 1008}, -3), ({"ldy": 63}, -3), ({"ldx": (1 << 30) + 8}, -3),
    ({"ldw": (1 << 30) + 16}, -3), ({"ldxq": (1 << 30) + 16}, -3), ({"ldy": (1 << 30) + 1}, -3),
    ({"x": A + 2}, -4), ({"ldx": 1028}, -4), ({"w13": A + 8}, -4), ({"ldw": 1032}, -4), ({"s13": A + 2}, -4),
    ({"xq": A + 8}, -4), ({"ldxq": 1032}, -4), ({"xs": A + 1}, -4), ({"y": A + 1}, -4)])
def test_glu_refusals(q, change, status):
    assert q.qlin_glu_i8(*{**GLU, **change}.values(), None) == status


MOE = dict(x=A, ldx=512, M=4, H=512, dtype=0, logits=A, ldl=8, E=8, topk=2, route=0, w13=A, ldw13=512, s13=A, I=128, w2=A,
           ldw2=128, s2=A, act=0, ids=A, gw=A, y=A, ldy=512, work=A, size=1 << 40)


@pytest.mark.parametrize("change,status", [
    ({"dtype": 2}, -6), ({"act": 2}, -6), ({"route": 2}, -6), ({"route": -1}, -6),
    ({"x": None}, -1), ({"w13": None}, -1), ({"s13": None}, -1), ({"w2": None}, -1), ({"s2": None}, -1), ({"ids": None}, -1),
    ({"gw": None}, -1), ({"y": None}, -1),
    ({"M": 0}, -2), ({"M": 16385}, -2), ({"H": 500}, -2), ({"H": 0}, -2), ({"H": 131088}, -2), ({"I": 8}, -2), ({"I": 120}, -2),
    ({"I": 131088}, -2), ({"E": 0}, -2), ({"E": 1025}, -2), ({"topk": 0}, -2), ({"topk": 17}, -2), ({"topk": 9}, -2),
    ({"topk": 17, "logits": None}, -2),
    ({"ldx": 504}, -3), ({"ldl": 7}, -3), ({"ldw13": 496}, -3), ({"ldw2": 112}, -3), ({"ldy": 511}, -3),
    ({"ldx": (1 << 30) + 8}, -3), ({"ldl": (1 << 30) + 1}, -3), ({"ldw13": (1 << 30) + 16}, -3), ({"ldw2": (1 << 30) + 16}, -3),
    ({"ldy": (1 << 30) + 1}, -3),
    ({"x": A + 8}, -4), ({"ldx": 516}, -4), ({"logits": A + 2}, -4), ({"w13": A + 4}, -4), ({"ldw13": 520}, -4),
    ({"s13": A + 1}, -4), ({"w2": A + 8}, -4), ({"ldw2": 136}, -4), ({"s2": A + 2}, -4), ({"ids": A + 2}, -4),
    ({"gw": A + 2}, -4), ({"y": A + 1}, -4), ({"work": None}, -5), ({"size": 64}, -5), ({"work": A + 8}, -4)])
def test_moe_refusals(q, change, status):
    assert q.qlin_moe_ffn_i8(*{**MOE, **change}.values(), None) == status


def test_moe_workspace(q):
    """One byte less than asked for is refused; sizes that the call refuses have none."""
    for M, H, I, topk, E in ((1, 16, 16, 1, 1), (4, 512, 128, 2, 8), (16, 7168, 2048, 6, 64), (1000, 2048, 768, 8, 128),
                             (16384, 16, 16, 16, 1024)):
        need = q.qlin_moe_ffn_i8_workspace_bytes(M, H, I, topk, E)
        assert need > M * topk * I * 2
        a = dict(MOE, M=M, H=H, I=I, topk=topk, E=E, ldx=H, ldl=E, ldw13=H, ldw2=I, ldy=H, logits=None)
        assert q.qlin_moe_ffn_i8(*{**a, "size": need - 1}.values(), None) == -5
    for bad in ((0, 512, 128, 2, 8), (4, 500, 128, 2, 8), (4, 512, 100, 2, 8), (4, 512, 128, 17, 8), (4, 512, 128, 2, 1025)):
        assert q.qlin_moe_ffn_i8_workspace_bytes(*bad) == 0


# ------------------------------------------------------------------ the definition itself

def test_quantiser_is_the_int8_rule(orc):
    """Codes and scales equal those of the INT8 quantiser's oracle, bit for bit."""
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((6, 256)) * 10.0 ** rng.integers(-30, 30, (6, 1))).astype(np.float32)
    x[3] = 0
    bits = (x.view(np.uint32) >> 16).astype(np.uint16)
    val = (bits.astype(np.uint32) << 16).view(np.float32)
    codes, scales = orc.act_quant_i8(bits)
    q, s = i8ffn.quantise(val)
    assert np.array_equal(q, codes.astype(np.float64)) and np.array_equal(s, scales.astype(np.float64))


def test_quantiser_without_finite_values():
    x = np.ones((3, 16))
    x[0, 3], x[1, 5] = np.inf, np.nan
    q, s = i8ffn.quantise(x)
    assert np.isnan(s[:2]).all() and (q[:2] == 0).all() and (q[2] == 127).all()


def test_routing_order_and_masks():
    lg = np.array([[1.0, 3.0, 3.0, -np.inf, np.nan, 2.0], [-np.inf] * 6, [0.0, -0.0, 0.0, -1.0, -1.0, -1.0],
                   [np.inf, 1.0, np.inf, 0.0, 0.0, 0.0], [np.nan, -np.inf, np.nan, -3e38, np.nan, np.nan]])
    ids, gw = i8ffn.route(lg, 4, 0)
    assert ids.tolist() == [[1, 2, 5, 0], [-1] * 4, [0, 1, 2, 3], [0, 2, 1, 3], [3, -1, -1, -1]]
    assert (gw[1] == 0).all() and gw[3].tolist() == [0.5, 0.5, 0.0, 0.0] and gw[4].tolist() == [1, 0, 0, 0]
    _, every = i8ffn.route(lg, 2, 1)
    e = np.exp(np.array([1.0, 3.0, 3.0, 2.0]) - 3.0)
    assert np.allclose(every[0], [1 / e.sum(), 1 / e.sum()])


def test_down_bounds_a_code_that_may_be_either():
    """A hidden value whose error reaches over the border of two 16-bit values moves its code: the bound covers it."""
    rng = np.random.default_rng(1)
    h = rng.standard_normal((1, 32))
    w, s2 = rng.integers(-128, 128, (8, 32)), np.full(8, 0.01)
    border = (i8ffn.round16(h, "bf16") + i8ffn.round16(h * (1 + 2.0 ** -7), "bf16")) / 2
    y0, _, t0 = i8ffn.down(h, np.zeros_like(h), w, s2, "bf16")
    assert (t0 == 0).all()
    y, _, tol = i8ffn.down(border, np.abs(border) * 2.0 ** -9, w, s2, "bf16")
    up, _, _ = i8ffn.down(border * (1 + 2.0 ** -8), np.zeros_like(h), w, s2, "bf16")
    assert (tol > 0).all() and (np.abs(up - y) <= tol * 1.01 + 1e-12).all()
