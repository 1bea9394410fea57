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


def test_more_gates_than_a_launch_has_threads(ql):
    """M * I past 2^32 with an odd I (one column a thread), in place: rows at both ends and across 2^32."""
    M, I, dt = 16384, (1 << 18) + 1, torch.bfloat16
    w, ws, wz = gen_w4(2 * I, 32, 32, "bf16", False, seed=1)
    layer = dev_w(w, ws, wz)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    buf = torch.empty((M, 2 * I + 6), dtype=dt, device="cuda").normal_(generator=gen)
    gu = buf[:, :2 * I]
    dy = torch.empty((M, I), dtype=dt, device="cuda").normal_(generator=gen)
    rows = [0, 1, 4095, 8191, 8192, M - 3, M - 2, M - 1]
    before, pads = gu[rows].double(), buf[:, 2 * I:].clone()
    _, dgu = ql.qlin_glu_w4_bwd(dy, *layer, gu=gu, dgu=gu, need_dx=False)
    assert dgu.data_ptr() == gu.data_ptr()
    g, u, d = before[:, :I], before[:, I:], dy[rows].double()
    s = torch.sigmoid(g)
    want = torch.cat((d * u * (s + g * s * (1 - s)), d * g * s), dim=1)
    # one rounding (2^-8) of a product of fp32 terms: 64 ulps of 2^-24 times |g| <= 6 stay below 2^-14 of |d u| or |d g|
    slack = torch.cat((d * u, d * g), dim=1).abs() * 2.0 ** -14
    got = dgu[rows].double()
    assert bool(((got - want).abs() <= want.abs() * 2.0 ** -8 + slack).all())
    assert torch.equal(buf[:, 2 * I:], pads)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M,N,groups", [(64, 100, 551), (50, 33, 896), (64, 70, 934), (64, 70, 935), (64, 65, 936), (48, 41, 810),
                                        (33, 64, 1100), (20, 100, 1270), (200, 70, 700)])
def test_rows_of_many_scales(ql, M, N, groups, dtype):
    """17 and more tokens, groups of 32: two stages next to the scales of 32 rows, on each side of the limits."""
    K = 32 * groups
    w, ws, wz = gen_w4(N, K, 32, dtype, True, seed=N, exact_scales=True)
    layer = dev_w(w, ws, wz)
    W, P = ref.dense(w, f64(ws), wz, 32), ref.dense_parts(w, f64(ws), wz, 32)
    x = gen_x(M, K, dtype, seed=M, scale=0.1)
    y, S, Q = ref.product(f64(x), W.T, P.T)
    E = ref.sum_tolerance(S, Q, K, dtype, True)
    close(ql.qlin_gemv_w4(x.cuda(), *layer), y, ref.rounded_tolerance(y, E, dtype), "y")
    if N % 2 == 0:
        gu = torch.empty((M, N), dtype=DT[dtype], device="cuda")
        ql.qlin_glu_w4(x.cuda(), *layer, gu=gu)
        close(gu, y, ref.rounded_tolerance(y, E, dtype), "gu")


def _one_weight(rows, dtype, code, zero, scale):
    """A layer whose weights are all scale * (code - zero)."""
    w = torch.full((rows, 32), code * 17, dtype=torch.uint8, device="cuda")
    ws = torch.full((rows, 2), scale, dtype=DT[dtype], device="cuda")
    return w, ws, torch.full((rows, 2), zero, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("M", [1, 9, 16, 17, 40, 300])
def test_weights_beyond_fp16(ql, M):
    """8000 * 15 is no fp16 number: without rounding a product of it is finite, with it infinite."""
    layer = _one_weight(72, "fp16", 15, 0, 8000.0)
    x = torch.full((M, 64), 2.0 ** -10, dtype=torch.float16, device="cuda")
    y = ql.qlin_gemv_w4(x, *layer)
    assert bool((y == (7500.0 if M <= 16 else float("inf"))).all())
    dx = ql.qlin_gemv_w4_bwd(torch.full((M, 72), 2.0 ** -10, dtype=torch.float16, device="cuda"), *layer)
    assert bool(torch.isinf(dx).all())


@pytest.mark.parametrize("M", [1, 9, 16, 17, 40, 300])
@pytest.mark.parametrize("code,zero", [(15, 0), (0, 15), (9, 8), (14, 15)])
def test_largest_bf16_scales(ql, M, code, zero):
    """Scales of 2^124: exact products with small activations, though zero * scale is close to fp32's end."""
    layer = _one_weight(72, "bf16", code, zero, 2.0 ** 124)
    x = torch.full((M, 64), 2.0 ** -100, dtype=torch.bfloat16, device="cuda")
    y = ql.qlin_gemv_w4(x, *layer)
    assert bool((y == (code - zero) * 2.0 ** 30).all())  # 64 * 2^124 * 2^-100
    dx = ql.qlin_gemv_w4_bwd(torch.full((M, 72), 2.0 ** -100, dtype=torch.bfloat16, device="cuda"), *layer)
    assert bool((dx == (code - zero) * 9 * 2.0 ** 27).all())
