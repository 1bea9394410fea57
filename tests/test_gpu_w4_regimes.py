"""The 4-bit weight operators in every kernel and layout that the sizes choose: the GEMM's two tiles, the decode
kernels' passes and rounds, blocks of 64 tokens, shares of the gradient; then random calls, and numbers that are
not finite."""
import numpy as np
import pytest
import torch

from gpu_util import lib, need_gpu
from oracle import w4 as ref
from w4_util import DT, close, dev_w, f64, gen_w4, gen_x, guards_intact, out_view, pitched

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def _mats(w, ws, wz, group):
    return ref.dense(w, f64(ws), wz, group), ref.dense_parts(w, f64(ws), wz, group)


def _linear(M, N, K, group, dtype, zeros, exact, seed, pads=(0, 0, 3), bias=False):
    """Forward and input gradient of one random layer."""
    ql = lib()
    xp, wp, yp = pads
    w, ws, wz = gen_w4(N, K, group, dtype, zeros, seed=seed, exact_scales=exact)
    x, dy = gen_x(M, K, dtype, seed + 1), gen_x(M, N, dtype, seed + 2)
    b = gen_x(1, N, dtype, seed + 3)[0] if bias else None
    wd, sd, zd = dev_w(w, ws, wz, pad=wp)
    W, P = _mats(w, ws, wz, group)
    yv, buf = out_view(M, N, dtype, pad=yp)
    ql.qlin_gemv_w4(pitched(x, xp), wd, sd, zd, bias=None if b is None else b.cuda(), y=yv)
    y, S, Q = ref.product(f64(x), W.T, P.T)
    if bias:
        y = y + f64(b)
    E = ref.sum_tolerance(S, Q, K, dtype, exact) + (2.0 ** -24 * np.abs(y) if bias else 0.0)
    close(yv, y, ref.rounded_tolerance(y, E, dtype), "y")
    guards_intact(buf, M, N)
    dv, buf = out_view(M, K, dtype, pad=yp)
    ql.qlin_gemv_w4_bwd(pitched(dy, xp), wd, sd, zd, dx=dv)
    y, S, Q = ref.product(f64(dy), W, P)
    E = ref.sum_tolerance(S, Q, N, dtype, exact)
    close(dv, y, ref.rounded_tolerance(y, E, dtype), "dx")
    guards_intact(buf, M, K)


# the GEMM's 128 x 128 tiles, its 256 x 256 tiles; one group a row, several to a 64-deep step, none a power of two
GEMM = [(130, 70000, 96, 32), (17, 200000, 64, 64), (300, 20000, 1056, 96), (2000, 9001, 160, 160),
        (600, 40001, 96, 32), (4096, 4100, 544, 32), (4000, 4097, 512, 512), (4090, 4099, 640, 128)]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M,N,K,group", GEMM)
def test_gemm_tiles(M, N, K, group, dtype, zeros):
    _linear(M, N, K, group, dtype, zeros, True, seed=M + N, pads=(8, 16, 3), bias=not zeros)


def test_gemm_rounded_weights():
    _linear(4080, 4111, 352, 32, "bf16", True, False, seed=1)
    _linear(4080, 4111, 384, 128, "fp16", False, False, seed=2)


# the decode kernels: rows walked in several passes, tails of every kind, groups of every fold unit, several rounds
LONG = [(M, N, K, group) for M in (1, 2, 5, 8, 11, 16)
        for N, K, group in [(40, 8224, 32), (33, 14336, 128), (17, 16448, 64), (24, 13824, 384), (9, 20480, 20480),
                            (4500, 2080, 160), (21000, 256, 256), (300, 28800, 96)]]


@pytest.mark.parametrize("M,N,K,group", LONG)
def test_long_rows(M, N, K, group):
    dtype = "bf16" if (M + N) % 2 else "fp16"
    _linear(M, N, K, group, dtype, M % 3 != 0, False, seed=M + K, pads=(8, 16, 1), bias=M % 2 == 0)


# 17 to 64 tokens and blocks of 64: one to four row tiles, K past the first steps, tails
MID = [(20, 30, 4128, 32), (32, 9000, 256, 32), (33, 17000, 128, 64), (64, 25000, 96, 96), (48, 33000, 64, 32),
       (61, 100, 8192, 128), (200, 500, 2304, 64), (1000, 60, 1056, 32)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M,N,K,group", MID)
def test_row_tiles(M, N, K, group, dtype):
    _linear(M, N, K, group, dtype, True, True, seed=M + N, pads=(16, 16, 2), bias=True)


def test_one_row_gradient_of_every_width():
    """Shares of the gradient: short and long N, K from one block of columns to many."""
    for M, N, K in [(1, 31, 32), (1, 5000, 32), (16, 4099, 96), (17, 1000, 8192), (64, 12345, 160), (33, 64, 20000),
                    (70, 9000, 64), (520, 5000, 320)]:
        _linear(M, N, K, 32, "bf16", True, True, seed=N)


def _glu(M, I, K, group, dtype, act, zeros, seed, keep):
    """Front and its gradients with exact weights: kept or recomputed gate and up."""
    ql = lib()
    w, ws, wz = gen_w4(2 * I, K, group, dtype, zeros, seed=seed, exact_scales=True)
    x, dy = gen_x(M, K, dtype, seed + 1, scale=2.0 / np.sqrt(K)), gen_x(M, I, dtype, seed + 2)
    wd, sd, zd = dev_w(w, ws, wz, pad=16)
    W, P = _mats(w, ws, wz, group)
    gv, gbuf = out_view(M, 2 * I, dtype, 5)
    yv, ybuf = out_view(M, I, dtype, 3)
    xd = pitched(x, 8)
    ql.qlin_glu_w4(xd, wd, sd, zd, act=act, y=yv, gu=gv if keep else None)
    gu, S, Q = ref.product(f64(x), W.T, P.T)
    E = ref.sum_tolerance(S, Q, K, dtype, True)
    if keep:
        close(gv, gu, ref.rounded_tolerance(gu, E, dtype), "gu")
        guards_intact(gbuf, M, 2 * I)
    g, u, Eg, Eu = gu[:, :I], gu[:, I:], E[:, :I], E[:, I:]
    a, da, Ea, Eda = ref.gate_tolerance(g, u, Eg, Eu, act)
    want = a * u
    err = Ea * (np.abs(u) + Eu) + np.abs(a) * Eu + np.abs(want) * 2.0 ** -23
    close(yv, want, ref.rounded_tolerance(want, err, dtype), "y")
    guards_intact(ybuf, M, I)
    if keep:  # the kernel reads gate and up as they were stored
        g, u, Eg, Eu = f64(gv)[:, :I], f64(gv)[:, I:], 0.0, 0.0
        a, da, Ea, Eda = ref.gate_tolerance(g, u, 0.0, 0.0, act)
    dv, dbuf = out_view(M, K, dtype, 1)
    kept = {"gu": gv} if keep else {"x": xd}
    dx, dgu = ql.qlin_glu_w4_bwd(dy.cuda() if I % 8 == 0 else pitched(dy, 0), wd, sd, zd, act=act, dx=dv, **kept)
    d = f64(dy)
    want = np.concatenate([d * u * da, d * a], axis=1)
    err = np.concatenate([np.abs(d) * (Eda * (np.abs(u) + Eu) + np.abs(da) * Eu), np.abs(d) * Ea], axis=1)
    close(dgu, want, ref.rounded_tolerance(want, err + np.abs(want) * 2.0 ** -22, dtype), "dgu")
    y, S, Q = ref.product(f64(dgu), W, P)
    close(dx, y, ref.rounded_tolerance(y, ref.sum_tolerance(S, Q, 2 * I, dtype, True), dtype), "dx")
    guards_intact(dbuf, M, K)


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("M,I,K,group", [(4096, 2051, 544, 32), (4000, 2048, 512, 128), (130, 35000, 96, 32),
                                         (1000, 9000, 160, 160), (1, 20, 16384, 128), (6, 2500, 2080, 32),
                                         (14, 77, 10240, 64), (16, 9000, 288, 96), (40, 4099, 1024, 64),
                                         (64, 600, 4096, 32), (25, 16000, 64, 32), (260, 130, 1280, 128)])
def test_glu_regimes(M, I, K, group, keep):
    _glu(M, I, K, group, "bf16" if keep else "fp16", M % 2, True, M + I, keep)
    if M < 1000:
        _glu(M, I, K, group, "fp16" if keep else "bf16", 1 - M % 2, False, M + I + 9, keep)


@pytest.mark.parametrize("seed", range(40))
def test_random_calls(seed):
    rng = np.random.default_rng(seed)
    M = int(rng.choice([rng.integers(1, 17), rng.integers(17, 65), rng.integers(65, 700)]))
    group = 32 * int(rng.choice([1, 1, 2, 3, 4, 4, 5, 8, 12]))
    K = group * int(rng.integers(1, max(2, int(rng.choice([500, 2500, 9000])) // group)))
    N = int(rng.integers(1, 3000))
    dtype = ("bf16", "fp16")[seed % 2]
    pads = (8 * int(rng.integers(0, 3)), 16 * int(rng.integers(0, 3)), int(rng.integers(0, 9)))
    _linear(M, N, K, group, dtype, bool(rng.integers(0, 2)), bool(rng.integers(0, 2)), seed, pads, bool(rng.integers(0, 2)))
    _glu(M, int(rng.integers(1, 900)), K, group, dtype, int(rng.integers(0, 2)), bool(rng.integers(0, 2)), seed,
         bool(rng.integers(0, 2)))


@pytest.mark.parametrize("M,N,K", [(1, 24, 512), (7, 40, 1056), (13, 40, 512), (40, 70, 800), (300, 90, 512),
                                   (4096, 4100, 544)])
def test_not_finite_stays_in_its_row(M, N, K):
    """A token with infinities or NaN, a row of weights with a NaN scale: nothing else changes."""
    ql = lib()
    w, ws, wz = gen_w4(N, K, 32, "bf16", True, seed=5)
    wd, sd, zd = dev_w(w, ws, wz)
    x, dy = gen_x(M, K, "bf16", 6).cuda(), pitched(gen_x(M, N, "bf16", 7), 0)
    y, dx = ql.qlin_gemv_w4(x, wd, sd, zd), ql.qlin_gemv_w4_bwd(dy, wd, sd, zd)
    m, n = M // 2, N // 3
    for v in (float("nan"), float("inf"), float("-inf")):
        x2, dy2 = x.clone(), pitched(dy, 0)
        x2[m, K - 1] = v
        dy2[m, N - 1] = v
        y2, dx2 = ql.qlin_gemv_w4(x2, wd, sd, zd), ql.qlin_gemv_w4_bwd(dy2, wd, sd, zd)
        keep = torch.arange(M) != m
        assert torch.equal(y2[keep], y[keep]) and torch.equal(dx2[keep], dx[keep])
        code = (w[:, -1] >> 4) != wz[:, -1]
        assert not bool(torch.isfinite(y2[m].cpu()[torch.from_numpy(code)]).any())
        assert not bool(torch.isfinite(dx2[m].cpu()[::2][torch.from_numpy((w[N - 1] & 15) != np.repeat(wz[N - 1], 16))]).any())
    s2 = sd.clone()
    s2[n, 0] = float("nan")
    y2, dx2 = ql.qlin_gemv_w4(x, wd, s2, zd), ql.qlin_gemv_w4_bwd(dy, wd, s2, zd)
    keep = torch.arange(N) != n
    assert torch.equal(y2[:, keep], y[:, keep]) and bool(torch.isnan(y2[:, n]).all())
    assert torch.equal(dx2[:, 32:], dx[:, 32:]) and bool(torch.isnan(dx2[:, :32]).all())


def test_same_results_every_time():
    """No atomics: a call repeated gives the same bits."""
    ql = lib()
    for M, N, K in [(1, 5000, 4096), (16, 3000, 8192), (50, 4000, 2048), (700, 4000, 1024)]:
        w, ws, wz = gen_w4(N, K, 128, "bf16", True, seed=5)
        wd, sd, zd = dev_w(w, ws, wz)
        x, dy = gen_x(M, K, "bf16", 6).cuda(), gen_x(M, N, "bf16", 7).cuda()
        a = (ql.qlin_gemv_w4(x, wd, sd, zd), ql.qlin_gemv_w4_bwd(dy, wd, sd, zd), ql.qlin_glu_w4(x, wd, sd, zd))
        for _ in range(5):
            b = (ql.qlin_gemv_w4(x, wd, sd, zd), ql.qlin_gemv_w4_bwd(dy, wd, sd, zd), ql.qlin_glu_w4(x, wd, sd, zd))
            assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("M", [1, 12, 40, 300])
def test_small_and_large_scales(M):
    """fp16 scales below its normal numbers, bf16 scales far from 1: weights that the type still holds exactly."""
    ql = lib()
    N, K, group = 40, 256, 64
    rng = np.random.default_rng(M)
    for dtype, unit, most in [("fp16", 2.0 ** -24, 40), ("bf16", 2.0 ** -100, 8), ("bf16", 2.0 ** 90, 8)]:
        w, _, wz = gen_w4(N, K, group, dtype, True, seed=M)
        ws = torch.from_numpy(unit * rng.integers(1, most, size=(N, K // group))).to(DT[dtype])
        x, dy = gen_x(M, K, dtype, 1), gen_x(M, N, dtype, 2)
        wd, sd, zd = dev_w(w, ws, wz)
        W, P = _mats(w, ws, wz, group)
        y, S, Q = ref.product(f64(x), W.T, P.T)
        close(ql.qlin_gemv_w4(x.cuda(), wd, sd, zd), y,
              ref.rounded_tolerance(y, ref.sum_tolerance(S, Q, K, dtype, True), dtype), "y")
        y, S, Q = ref.product(f64(dy), W, P)
        close(ql.qlin_gemv_w4_bwd(dy.cuda(), wd, sd, zd), y,
              ref.rounded_tolerance(y, ref.sum_tolerance(S, Q, N, dtype, True), dtype), "dx")


@pytest.mark.parametrize("act", [0, 1])
def test_large_gates(act):
    """Gates far out on both sides: act is g or 0, act' is 1 or 0, nothing overflows on the way."""
    ql = lib()
    M, I, K = 3, 40, 64
    w, ws, wz = gen_w4(2 * I, K, 32, "bf16", True, seed=1)
    wd, sd, zd = dev_w(w, ws, wz)
    gu = torch.ones((M, 2 * I), dtype=torch.bfloat16)
    gates = [1e4, 1e10, 1e20, 1e30, 2.0 ** 126, -1e4, -1e10, -1e20, -1e30, -2.0 ** 126]
    gu[:, :I] = torch.tensor(gates * 4)
    dy = gen_x(M, I, "bf16", 2)
    _, dgu = ql.qlin_glu_w4_bwd(dy.cuda(), wd, sd, zd, act=act, gu=gu.cuda(), need_dx=False)
    dgu, up = dgu.cpu(), gu[:, :I] > 0
    assert torch.equal(dgu[:, :I], torch.where(up, dy, torch.zeros_like(dy)))
    want = torch.where(up, (dy.float() * gu[:, :I].float()).to(torch.bfloat16), torch.zeros_like(dy))
    assert torch.equal(dgu[:, I:], want)
