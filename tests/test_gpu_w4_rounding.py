"""What the 4-bit weight calls round, bit for bit.

Every scale is s, 2 s or 4 s with all of the type's digits in s, and x holds 64 values of -1 and 1 in each row, so
every partial sum of code * x or zero * x times a scale is a multiple of s below 64 * 15 * 2 * 4 = 7680 s: with the 11
digits of an fp16 s at most 24 bits, exact in fp32 in whatever order.  Where the weights are not rounded the result
is therefore r16(exact); where each is rounded first it is r16(sum of the rounded ones), which is exact in fp32 too
(multiples of the smallest weight's last digit, 2^-2 s / 2^10, below 2^13 s).  The two differ in many places."""
import numpy as np
import pytest
import torch

from gpu_util import lib, need_gpu
from oracle import w4 as ref
from w4_util import DT, f64

pytestmark = pytest.mark.gpu

UNIT = {"bf16": 173.0 / 128.0 / 16.0, "fp16": 1381.0 / 1024.0 / 16.0}  # s: an odd number of 8 or 11 binary digits


@pytest.fixture(scope="module")
def ql():
    need_gpu()
    return lib()


def _r16(v, dtype):
    t = torch.from_numpy(v).float()
    assert np.array_equal(t.double().numpy(), v)  # exact in fp32
    return t.to(DT[dtype])


def _sparse(rows, cols, rng):
    """64 values of -1 and 1 a row, its ends among them."""
    x = np.zeros((rows, cols))
    for r in x:
        at = rng.choice(cols, size=min(cols, 62), replace=False)
        r[at] = rng.choice([-1.0, 1.0], size=len(at))
        r[[0, cols - 1]] = rng.choice([-1.0, 1.0], size=2)
    return x


def _layer(rows, K, group, dtype, zeros, rng):
    w = rng.integers(0, 256, size=(rows, K // 2), dtype=np.uint8)
    ws = UNIT[dtype] * 2.0 ** rng.integers(0, 3, size=(rows, K // group))
    wz = rng.integers(0, 16, size=ws.shape, dtype=np.uint8) if zeros else None
    W = ref.dense(w, ws, wz, group)
    dev = (torch.from_numpy(w).cuda(), torch.from_numpy(ws).to(DT[dtype]).cuda(),
           None if wz is None else torch.from_numpy(wz).cuda())
    assert np.array_equal(f64(dev[1]), ws)
    return dev, W, f64(torch.from_numpy(W).to(DT[dtype]))


def _both(x, W, R, dtype):
    """(weights as they are, weights rounded first); the two can be told apart."""
    a, b = _r16(x @ W, dtype), _r16(x @ R, dtype)
    assert float((a != b).float().mean()) > 0.1
    return a, b


def _check(ql, M, rows, K, group, dtype, zeros, rounded, gated):
    rng = np.random.default_rng(M * 7 + rows + K)
    dev, W, R = _layer(rows, K, group, dtype, zeros, rng)
    x = _sparse(M, K, rng)
    xd = torch.from_numpy(x).to(DT[dtype]).cuda()
    want = _both(x, W.T, R.T, dtype)[rounded]
    if gated:
        got = torch.empty((M, rows), dtype=DT[dtype], device="cuda")
        ql.qlin_glu_w4(xd, *dev, gu=got)
    else:
        got = ql.qlin_gemv_w4(xd, *dev)
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M", list(range(1, 17)))
def test_decode_rounds_no_weight(ql, M, dtype, gated):
    for i, (rows, K, group) in enumerate([(66, 1024, 128), (130, 4480, 64), (24, 8224, 32), (40, 20480, 160),
                                          (4500, 288, 96), (18, 1 << 16, 1 << 16)]):
        _check(ql, M, rows, K, group, dtype, (i + M) % 2 == 0, False, gated)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M", [17, 33, 50, 70, 300, 700])
def test_more_tokens_round_each_weight_once(ql, M, dtype, gated):
    for i, (rows, K, group) in enumerate([(66, 1024, 128), (130, 4480, 64), (24, 8224, 32), (520, 288, 96)]):
        _check(ql, M, rows, K, group, dtype, (i + M) % 2 == 0, True, gated)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M,groups,gated", [(1, 5300, False), (8, 5300, False), (9, 2600, False), (16, 2600, False),
                                            (1, 2600, True), (8, 2600, True), (9, 1290, True), (16, 1290, True)])
def test_longest_rows_without_rounding(ql, M, groups, gated, dtype):
    """The most groups a row that the header names."""
    _check(ql, M, 24, 32 * groups, 32, dtype, M % 2 == 0, False, gated)
    _check(ql, M, 24, 64 * groups, 64, dtype, True, False, gated)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M,groups,gated", [(1, 6700, False), (8, 5400, False), (9, 2960, False), (16, 2680, False),
                                            (1, 3320, True), (8, 2680, True), (9, 1470, True), (16, 1320, True)])
def test_longer_rows_round(ql, M, groups, gated, dtype):
    """Rows of more scales than the decode kernels hold: each weight is rounded once."""
    _check(ql, M, 24, 32 * groups, 32, dtype, True, True, gated)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M", [1, 16, 17, 33, 64, 65, 300, 700])
def test_gradient_rounds_each_weight_once(ql, M, dtype):
    rng = np.random.default_rng(M)
    for rows, K, group in [(1000, 160, 32), (72, 1024, 128), (4099, 96, 96)]:
        dev, W, R = _layer(rows, K, group, dtype, rows == 72, rng)
        dy = _sparse(M, rows, rng)
        want = _both(dy, W, R, dtype)[1]
        pad = torch.zeros((M, (rows + 7) // 8 * 8), dtype=DT[dtype], device="cuda")
        pad[:, :rows] = torch.from_numpy(dy).to(DT[dtype])
        assert torch.equal(ql.qlin_gemv_w4_bwd(pad[:, :rows], *dev).cpu(), want)
