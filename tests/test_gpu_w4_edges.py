"""Ends of the value ranges of the 4-bit weight calls: gates that the 16-bit type holds as infinities."""
import numpy as np
import pytest
import torch

from gpu_util import lib, need_gpu
from oracle import w4 as ref
from w4_util import DT, close, dev_w, f64, gen_w4, gen_x

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ql():
    need_gpu()
    return lib()


@pytest.mark.parametrize("I", [40, 41])  # eight columns a thread, and one
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("act", [0, 1])
def test_kept_infinite_gates(ql, act, dtype, I):
    """act(-inf) = act'(-inf) = 0, act(inf) = inf and act'(inf) = 1; a NaN gate stays one."""
    inf = float("inf")
    w, ws, wz = gen_w4(2 * I, 64, 32, dtype, True, seed=1)
    layer = dev_w(w, ws, wz)
    gu = gen_x(4, 2 * I, dtype, 3)
    gu[0, :I], gu[1, :I], gu[2, :I] = -inf, inf, float("nan")
    dy = gen_x(4, I, dtype, 2)
    _, dgu = ql.qlin_glu_w4_bwd(dy.cuda(), *layer, act=act, gu=gu.cuda(), need_dx=False)
    dgu, u = dgu.cpu(), gu[:, I:]
    assert bool((dgu[0] == 0).all())
    assert torch.equal(dgu[1, :I], (dy[1].float() * u[1].float()).to(DT[dtype]))
    assert torch.equal(dgu[1, I:], dy[1].float().mul(inf).to(DT[dtype]))
    assert bool(torch.isnan(dgu[2]).all())
    assert bool(torch.isfinite(dgu[3].float()).all())


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("M", [1, 9, 40, 300, 2100])
def test_gates_below_the_lowest_fp16(ql, M, act):
    """Gates of -131072, which fp16 keeps as -inf: the output is 0 and so are both gradients, in every kernel."""
    I, K = 520, 64
    w = np.full((2 * I, K // 2), 0x77, np.uint8)           # codes 7: weights -scale
    w[::3] = 0x99                                          # codes 9: +scale
    w[:I] = 0x77
    ws = torch.full((2 * I, 2), 0.25, dtype=torch.float16)
    ws[:I] = 64.0
    layer = dev_w(w, ws, None)
    x = torch.full((M, K), 32.0, dtype=torch.float16, device="cuda")  # g = -64 * 32 * 64, u = +-512
    dy = gen_x(M, I, "fp16", 2).cuda()
    gu = torch.empty((M, 2 * I), dtype=torch.float16, device="cuda")
    y = ql.qlin_glu_w4(x, *layer, act=act, gu=gu)
    assert bool((gu[:, :I] == float("-inf")).all()) and bool((gu[:, I:].abs() == 512).all())
    assert bool((y == 0).all())
    for kept in ({"gu": gu}, {"x": x}):
        dx, dgu = ql.qlin_glu_w4_bwd(dy, *layer, act=act, **kept)
        assert bool((dgu == 0).all()) and bool((dx == 0).all())
