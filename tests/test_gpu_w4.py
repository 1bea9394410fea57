"""4-bit weight operators on the GPU against their plain 64-bit forms."""
import numpy as np
import pytest
import torch

from gpu_util import lib, need_gpu
from oracle import w4 as ref
from w4_util import DT, close, dev_w, f64, gen_w4, gen_x, guards_intact, out_view, pitched

pytestmark = pytest.mark.gpu

# (M, N, K, group): one token to a prompt, one row to many, one group to many, K that ends inside every
# tile depth, each side of the kernels' token limits
LINEAR = [(1, 1, 32, 32), (1, 16, 64, 64), (1, 17, 128, 128), (1, 1024, 1024, 128), (2, 33, 160, 32),
          (3, 100, 448, 64), (4, 64, 2048, 128), (5, 259, 1376, 32), (8, 48, 1024, 1024), (9, 130, 384, 96),
          (15, 31, 640, 128), (16, 256, 512, 64), (17, 65, 96, 32), (31, 200, 352, 32), (32, 72, 256, 128),
          (33, 129, 736, 32), (48, 96, 1024, 64), (64, 128, 128, 64), (65, 127, 192, 64), (100, 300, 224, 32),
          (129, 257, 320, 160), (300, 40, 1152, 128), (513, 270, 288, 32), (700, 513, 160, 32)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def _mats(w, ws, wz, group, transposed=False):
    W, parts = ref.dense(w, f64(ws), wz, group), ref.dense_parts(w, f64(ws), wz, group)
    return (W.T, parts.T) if transposed else (W, parts)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,N,K,group", LINEAR)
def test_linear(M, N, K, group, dtype, zeros):
    ql = lib()
    for exact in (True, False):
        w, ws, wz = gen_w4(N, K, group, dtype, zeros, seed=M + N + K, exact_scales=exact)
        x = gen_x(M, K, dtype, seed=M + K)
        bias = gen_x(1, N, dtype, seed=7)[0] if exact else None
        wd, wsd, wzd = dev_w(w, ws, wz, pad=0 if exact else 16)
        yv, buf = out_view(M, N, dtype, pad=3)
        got = ql.qlin_gemv_w4(pitched(x, 0 if exact else 8), wd, wsd, wzd,
                              bias=None if bias is None else bias.cuda(), y=yv)
        torch.cuda.synchronize()
        y, S, Q = ref.product(f64(x), *_mats(w, ws, wz, group, True))
        if bias is not None:
            y = y + f64(bias)
        E = ref.sum_tolerance(S, Q, K, dtype, exact)
        close(got, y, ref.rounded_tolerance(y, E, dtype), f"linear exact_scales={exact}")
        guards_intact(buf, M, N)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,N,K,group", LINEAR)
def test_linear_bwd(M, N, K, group, dtype, zeros):
    ql = lib()
    for exact in (True, False):
        w, ws, wz = gen_w4(N, K, group, dtype, zeros, seed=M + N + K, exact_scales=exact)
        dy = gen_x(M, N, dtype, seed=M + N)
        wd, wsd, wzd = dev_w(w, ws, wz, pad=0 if exact else 16)
        dxv, buf = out_view(M, K, dtype, pad=3)
        got = ql.qlin_gemv_w4_bwd(pitched(dy, 0 if exact else 8), wd, wsd, wzd, dx=dxv)
        torch.cuda.synchronize()
        y, S, Q = ref.product(f64(dy), *_mats(w, ws, wz, group))
        E = ref.sum_tolerance(S, Q, N, dtype, exact)
        close(got, y, ref.rounded_tolerance(y, E, dtype), f"input gradient exact_scales={exact}")
        guards_intact(buf, M, K)


def test_linear_bwd_long_reduction():
    """Many rows, few columns: the reduction over N is split, in order."""
    ql = lib()
    for M, N, K, dtype in [(1, 5003, 64, "bf16"), (7, 4096, 256, "fp16"), (70, 6400, 96, "fp16"),
                           (130, 3001, 128, "bf16")]:
        w, ws, wz = gen_w4(N, K, 32, dtype, True, seed=N, exact_scales=True)
        dy = gen_x(M, N, dtype, seed=N)
        wd, wsd, wzd = dev_w(w, ws, wz)
        dyd = pitched(dy, 0)
        got = ql.qlin_gemv_w4_bwd(dyd, wd, wsd, wzd)
        again = ql.qlin_gemv_w4_bwd(dyd, wd, wsd, wzd)
        torch.cuda.synchronize()
        y, S, Q = ref.product(f64(dy), *_mats(w, ws, wz, 32))
        close(got, y, ref.rounded_tolerance(y, ref.sum_tolerance(S, Q, N, dtype, True), dtype), f"{M}x{N}x{K}")
        assert torch.equal(got, again)


# (M, I, K, group)
GLU = [(1, 1, 32, 32), (1, 17, 128, 64), (1, 512, 1024, 128), (3, 40, 160, 32), (7, 33, 448, 64), (16, 96, 512, 128),
       (17, 31, 96, 32), (40, 65, 352, 32), (64, 64, 256, 256), (65, 100, 192, 64), (130, 129, 320, 160),
       (513, 200, 288, 32)]


def _glu_ref(x, mats, I):
    gu, S, Q = ref.product(x, mats[0].T, mats[1].T)
    return gu[:, :I], gu[:, I:], S, Q


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("M,I,K,group", GLU)
def test_glu(M, I, K, group, dtype, act):
    ql = lib()
    for exact in (True, False):
        w, ws, wz = gen_w4(2 * I, K, group, dtype, exact, seed=M + I, exact_scales=exact)
        x = gen_x(M, K, dtype, seed=M + K, scale=0.3)
        wd, wsd, wzd = dev_w(w, ws, wz, pad=0 if exact else 16)
        yv, ybuf = out_view(M, I, dtype, pad=5)
        gv, gbuf = out_view(M, 2 * I, dtype, pad=5)
        ql.qlin_glu_w4(pitched(x, 8), wd, wsd, wzd, act=act, y=yv, gu=gv)
        y2 = ql.qlin_glu_w4(pitched(x, 8), wd, wsd, wzd, act=act)
        torch.cuda.synchronize()
        g, u, S, Q = _glu_ref(f64(x), _mats(w, ws, wz, group), I)
        E = ref.sum_tolerance(S, Q, K, dtype, exact)
        Eg, Eu = E[:, :I], E[:, I:]
        a, _, Ea, _ = ref.gate_tolerance(g, u, Eg, Eu, act)
        close(yv, a * u, ref.rounded_tolerance(a * u, Ea * (np.abs(u) + Eu) + np.abs(a) * Eu, dtype), "y")
        gu = np.concatenate([g, u], axis=1)
        close(gv, gu, ref.rounded_tolerance(gu, E, dtype), "gu")
        assert torch.equal(yv, y2)
        guards_intact(ybuf, M, I)
        guards_intact(gbuf, M, 2 * I)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("M,I,K,group", GLU)
def test_glu_bwd(M, I, K, group, act, keep, dtype):
    ql = lib()
    w, ws, wz = gen_w4(2 * I, K, group, dtype, keep, seed=M + I, exact_scales=True)
    mats = _mats(w, ws, wz, group)
    wd, wsd, wzd = dev_w(w, ws, wz, pad=16)
    dy = gen_x(M, I, dtype, seed=5)
    x = gen_x(M, K, dtype, seed=M + K, scale=0.3)
    gu16 = gen_x(M, 2 * I, dtype, seed=6, scale=2.0)
    dgu, gbuf = out_view(M, 2 * I, dtype, pad=8 + (-2 * I) % 8)
    dxv, xbuf = out_view(M, K, dtype, pad=3)
    kw = {"gu": pitched(gu16, 1, multiple=1)} if keep else {"x": pitched(x, 8)}
    ql.qlin_glu_w4_bwd(pitched(dy, 1, multiple=1), wd, wsd, wzd, act=act, dgu=dgu, dx=dxv, **kw)
    torch.cuda.synchronize()
    if keep:
        g, u = f64(gu16)[:, :I], f64(gu16)[:, I:]
        Eg = Eu = np.zeros_like(g)
    else:
        g, u, S, Q = _glu_ref(f64(x), mats, I)
        E = ref.sum_tolerance(S, Q, K, dtype, True)
        Eg, Eu = E[:, :I], E[:, I:]
    a, da, Ea, Eda = ref.gate_tolerance(g, u, Eg, Eu, act)
    d = f64(dy)
    want = np.concatenate([d * u * da, d * a], axis=1)
    err = np.concatenate([np.abs(d) * ((np.abs(u) + Eu) * Eda + Eu * np.abs(da)) + np.abs(want[:, :I]) * 2.0 ** -22,
                          np.abs(d) * Ea + np.abs(want[:, I:]) * 2.0 ** -22], axis=1)
    close(dgu, want, ref.rounded_tolerance(want, err, dtype), "dgu")
    guards_intact(gbuf, M, 2 * I)
    # the second product, from the 16-bit dgu that the call wrote
    y, S, Q = ref.product(f64(dgu), *mats)
    close(dxv, y, ref.rounded_tolerance(y, ref.sum_tolerance(S, Q, 2 * I, dtype, True), dtype), "dx")
    guards_intact(xbuf, M, K)


def test_glu_bwd_in_place_and_without_dx():
    """dgu may be gu itself; need_dx=False computes dgu only."""
    ql = lib()
    w, ws, wz = gen_w4(128, 256, 64, "bf16", True, seed=1)
    wd, wsd, wzd = dev_w(w, ws, wz)
    dy, gu = gen_x(9, 64, "bf16", 2).cuda(), gen_x(9, 128, "bf16", 3).cuda()
    dx, dgu = ql.qlin_glu_w4_bwd(dy, wd, wsd, wzd, gu=gu)
    none, dgu2 = ql.qlin_glu_w4_bwd(dy, wd, wsd, wzd, gu=gu, need_dx=False)
    kept = gu.clone()
    dx3, dgu3 = ql.qlin_glu_w4_bwd(dy, wd, wsd, wzd, gu=kept, dgu=kept)
    torch.cuda.synchronize()
    assert none is None and torch.equal(dgu, dgu2) and torch.equal(dgu, dgu3) and torch.equal(dx, dx3)
    assert dgu3.data_ptr() == kept.data_ptr()
