"""The 4-bit weight operators as programs use them: captured graphs, other streams, several threads, autograd,
a whole feed-forward block, very long rows and matrices past 4 GiB."""
import threading

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
    import skinny_gemm_qlin_amd.torch_ops  # noqa: F401
    return lib()


def _mats(w, ws, wz, group):
    return ref.dense(w, f64(ws), wz, group), ref.dense_parts(w, f64(ws), wz, group)


def _replay(step, feeds):
    """Captures step() once and compares replays with fresh inputs with eager calls, bit for bit."""
    step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for feed in feeds:
        feed()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        eager = [o.clone() for o in step()]
        torch.cuda.synchronize()
        for a, b in zip(got, eager):
            assert torch.equal(a, b)


@pytest.mark.parametrize("M", [1, 12, 40, 100, 600])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_graphs(ql, M, dtype):
    """Every entry point, in each regime of M; the workspace is the caller's."""
    I, K, G = 96, 512, 64
    w, ws, wz = gen_w4(2 * I, K, G, dtype, True, seed=M)
    wd, sd, zd = dev_w(w, ws, wz)
    x, dy = gen_x(M, K, dtype, 1).cuda(), gen_x(M, I, dtype, 2).cuda()
    gu = torch.empty((M, 2 * I), dtype=DT[dtype], device="cuda")
    dgu, dx, dx2 = torch.empty_like(gu), torch.empty_like(x), torch.empty_like(x)
    y, y2 = torch.empty((M, I), dtype=DT[dtype], device="cuda"), torch.empty((M, 2 * I), dtype=DT[dtype], device="cuda")
    need = ql.qlin_gemv_w4_bwd_workspace_bytes(M, 2 * I, K)
    work = torch.empty((max(need, 16),), dtype=torch.uint8, device="cuda")

    def step():
        ql.qlin_gemv_w4(x, wd, sd, zd, y=y2)
        ql.qlin_glu_w4(x, wd, sd, zd, act=1, y=y, gu=gu)
        ql.qlin_glu_w4_bwd(dy, wd, sd, zd, act=1, gu=gu, dgu=dgu, dx=dx, workspace=work)
        ql.qlin_glu_w4_bwd(dy, wd, sd, zd, act=1, x=x, dgu=dgu, dx=dx2, workspace=work)
        return y2, y, gu, dgu, dx, dx2

    def feed(seed):
        def f():
            x.copy_(gen_x(M, K, dtype, seed))
            dy.copy_(gen_x(M, I, dtype, seed + 1))
            work.fill_(255)  # what it holds on entry does not matter
        return f

    _replay(step, [feed(s) for s in (11, 22, 33, 44)])


def test_forward_and_backward_in_a_graph(ql):
    """A training step through autograd, captured; an eager graph of the same leaf is gone by then."""
    w, ws, wz = gen_w4(256, 128, 32, "bf16", True, seed=3)
    wd, sd, zd = dev_w(w, ws, wz)
    w2, ws2, _ = gen_w4(128, 128, 128, "bf16", False, seed=4)
    wd2, sd2, _ = dev_w(w2, ws2, None)
    x = gen_x(70, 128, "bf16", 5).cuda().requires_grad_(True)
    dout = gen_x(70, 128, "bf16", 6).cuda()

    def step():
        y, _ = torch.ops.qlin.glu_w4(x, wd, sd, zd, 0, True)
        out = torch.ops.qlin.gemv_w4(y, wd2, sd2)
        (dx,) = torch.autograd.grad(out, x, dout)
        return out.detach(), dx

    def feed(seed):
        def f():
            with torch.no_grad():
                x.copy_(gen_x(70, 128, "bf16", seed))
        return f

    _replay(step, [feed(s) for s in (7, 8, 9)])


def test_autograd(ql):
    """torch.ops.qlin: gradients equal the direct calls; expanded and transposed gradients; frozen weights."""
    M, I, K = 33, 50, 96
    w, ws, wz = gen_w4(2 * I, K, 32, "fp16", True, seed=1)
    wd, sd, zd = dev_w(w, ws, wz)
    x = gen_x(M, K, "fp16", 2).cuda().requires_grad_(True)
    out = torch.ops.qlin.gemv_w4(x, wd, sd, zd)
    assert torch.equal(out, ql.qlin_gemv_w4(x.detach(), wd, sd, zd))
    ones = torch.ones_like(out)
    (g1,) = torch.autograd.grad(out.sum(), x)            # the gradient of out is an expanded scalar
    assert torch.equal(g1, ql.qlin_gemv_w4_bwd(torch.ops.aten.constant_pad_nd(ones, (0, 4))[:, :2 * I], wd, sd, zd))
    back = gen_x(2 * I, M, "fp16", 3).cuda()
    out = torch.ops.qlin.gemv_w4(x, wd, sd, zd)
    (g2,) = torch.autograd.grad(out.t(), x, back)        # a transposed one
    pad = torch.zeros((M, 2 * I + 4), dtype=torch.float16, device="cuda")
    pad[:, :2 * I] = back.t()
    assert torch.equal(g2, ql.qlin_gemv_w4_bwd(pad[:, :2 * I], wd, sd, zd))
    dy = gen_x(M, I, "fp16", 4).cuda()
    for keep in (False, True):
        y, gu = torch.ops.qlin.glu_w4(x, wd, sd, zd, 1, keep)
        (gx,) = torch.autograd.grad(y, x, dy)
        dx, _ = ql.qlin_glu_w4_bwd(dy, wd, sd, zd, act=1, **({"gu": gu.detach()} if keep else {"x": x.detach()}))
        assert torch.equal(gx, dx)
    with pytest.raises(RuntimeError, match="frozen"):
        torch.ops.qlin.gemv_w4(x, wd, sd.clone().requires_grad_(True), zd)
    y, gu = torch.ops.qlin.glu_w4(x, wd, sd, zd, 0, True)
    with pytest.raises(RuntimeError, match="gradient of its own"):
        gu.sum().backward()
    torch.library.opcheck(torch.ops.qlin.gemv_w4.default, (x.detach(), wd, sd, zd),
                          test_utils=("test_schema", "test_faketensor"))
    torch.library.opcheck(torch.ops.qlin.glu_w4.default, (x.detach(), wd, sd, zd, 1, True),
                          test_utils=("test_schema", "test_faketensor"))


@pytest.mark.parametrize("M", [1, 20, 130])
def test_feed_forward_block(ql, M):
    """gate/up, down, and back through both: each stage against the exact product of what the one before wrote."""
    dtype, H, I, G = "bf16", 256, 200, 32
    w13, s13, z13 = gen_w4(2 * I, H, G, dtype, True, seed=M, exact_scales=True)
    w2, s2, _ = gen_w4(H, 224, G, dtype, False, seed=M + 1, exact_scales=True)  # I padded to a multiple of 32
    a, b = dev_w(w13, s13, z13), dev_w(w2, s2, None)
    x = gen_x(M, H, dtype, 5, scale=0.3).cuda()
    act = torch.zeros((M, 224), dtype=DT[dtype], device="cuda")
    gu = torch.empty((M, 2 * I), dtype=DT[dtype], device="cuda")
    ql.qlin_glu_w4(x, *a, y=act[:, :I], gu=gu)
    out = ql.qlin_gemv_w4(act, *b)
    dout = gen_x(M, H, dtype, 6).cuda()
    dact = ql.qlin_gemv_w4_bwd(dout, *b)
    dx, dgu = ql.qlin_glu_w4_bwd(dact[:, :I], *a, gu=gu)
    torch.cuda.synchronize()
    W13, P13 = _mats(w13, s13, z13, G)
    W2, P2 = _mats(w2, s2, None, G)
    for got, left, W, P, R in [(gu, x, W13.T, P13.T, H), (out, act, W2.T, P2.T, 224), (dact, dout, W2, P2, H),
                               (dx, dgu, W13, P13, 2 * I)]:
        y, S, Q = ref.product(f64(left), W, P)
        close(got, y, ref.rounded_tolerance(y, ref.sum_tolerance(S, Q, R, dtype, True), dtype), "stage")
    g, u, d = f64(gu)[:, :I], f64(gu)[:, I:], f64(dact)[:, :I]
    ga, gda, Ea, Eda = ref.gate_tolerance(g, u, 0.0, 0.0, 0)
    want = np.concatenate([d * u * gda, d * ga], axis=1)
    err = np.concatenate([np.abs(d * u) * Eda, np.abs(d) * Ea], axis=1) + np.abs(want) * 2.0 ** -22
    close(dgu, want, ref.rounded_tolerance(want, err, dtype), "dgu")


def test_streams_and_threads(ql):
    """Calls on several streams from several threads, each with its own buffers, equal the serial ones."""
    K, I = 1024, 160
    w, ws, wz = gen_w4(2 * I, K, 128, "bf16", True, seed=9)
    wd, sd, zd = dev_w(w, ws, wz)
    jobs = [(M, gen_x(M, K, "bf16", M).cuda(), gen_x(M, 2 * I, "bf16", M + 1).cuda()) for M in (1, 5, 14, 33, 80, 300)]
    want = [(ql.qlin_gemv_w4(x, wd, sd, zd), ql.qlin_glu_w4(x, wd, sd, zd), ql.qlin_gemv_w4_bwd(dy, wd, sd, zd))
            for _, x, dy in jobs]
    torch.cuda.synchronize()
    got, errors = [None] * len(jobs), []

    def run(i):
        try:
            _, x, dy = jobs[i]
            st = torch.cuda.Stream()
            outs = None
            for _ in range(20):
                with torch.cuda.stream(st):
                    outs = (ql.qlin_gemv_w4(x, wd, sd, zd), ql.qlin_glu_w4(x, wd, sd, zd),
                            ql.qlin_gemv_w4_bwd(dy, wd, sd, zd))
            st.synchronize()
            got[i] = outs
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for a, b in zip(got, want):
        for p, q in zip(a, b):
            assert torch.equal(p, q)


def test_stream_argument(ql):
    """`stream` takes a torch stream or its raw handle; a raw one needs a workspace of the caller's."""
    w, ws, wz = gen_w4(2048, 64, 32, "bf16", True, seed=2)
    wd, sd, zd = dev_w(w, ws, wz)
    x, dy = gen_x(3, 64, "bf16", 1).cuda(), gen_x(3, 2048, "bf16", 2).cuda()
    want, wantd = ql.qlin_gemv_w4(x, wd, sd, zd), ql.qlin_gemv_w4_bwd(dy, wd, sd, zd)
    y, dx = torch.empty_like(want), torch.empty_like(wantd)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    ql.qlin_gemv_w4(x, wd, sd, zd, y=y, stream=st)
    ql.qlin_gemv_w4_bwd(dy, wd, sd, zd, dx=dx, stream=st)
    st.synchronize()
    assert torch.equal(y, want) and torch.equal(dx, wantd)
    y.zero_()
    torch.cuda.synchronize()
    ql.qlin_gemv_w4(x, wd, sd, zd, y=y, stream=st.cuda_stream)
    st.synchronize()
    assert torch.equal(y, want)
    need = ql.qlin_gemv_w4_bwd_workspace_bytes(3, 2048, 64)
    assert need > 0
    with pytest.raises(ValueError, match="workspace"):
        ql.qlin_gemv_w4_bwd(dy, wd, sd, zd, dx=dx, stream=st.cuda_stream)
    with pytest.raises(ql.QlinError, match="WORKSPACE"):
        ql.qlin_gemv_w4_bwd(dy, wd, sd, zd, dx=dx, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("M,N,K,group", [(1, 24, 65536, 128), (8, 16, 40960, 32), (16, 20, 20480, 64), (3, 8, 262144, 32),
                                         (30, 9, 262144, 32), (2, 5, 1 << 20, 1 << 20), (16384, 3, 32, 32),
                                         (16384, 40, 64, 32), (5, 40000, 256, 64), (70, 2, 4096, 4096)])
def test_extreme_sizes(ql, M, N, K, group):
    """Rows walked in many passes, more scales than LDS holds, the most tokens, very tall and very flat matrices."""
    w, ws, wz = gen_w4(N, K, group, "fp16", True, seed=N, exact_scales=True)
    x = gen_x(M, K, "fp16", seed=1, scale=0.05)
    wd, sd, zd = dev_w(w, ws, wz)
    got = ql.qlin_gemv_w4(x.cuda(), wd, sd, zd)
    W, P = _mats(w, ws, wz, group)
    y, S, Q = ref.product(f64(x), W.T, P.T)
    close(got, y, ref.rounded_tolerance(y, ref.sum_tolerance(S, Q, K, "fp16", True), "fp16"), "y")
    dy = gen_x(M, N, "fp16", seed=3)
    pad = torch.zeros((M, (N + 7) // 8 * 8), dtype=torch.float16, device="cuda")
    pad[:, :N] = dy.cuda()
    gotd = ql.qlin_gemv_w4_bwd(pad[:, :N], wd, sd, zd)
    y, S, Q = ref.product(f64(dy), W, P)
    close(gotd, y, ref.rounded_tolerance(y, ref.sum_tolerance(S, Q, N, "fp16", True), "fp16"), "dx")


def test_past_32_bits(ql):
    """A code matrix of 4.9 GB: rows at both ends, forward in every regime and backward."""
    N, K, G, T = 600_000, 16384, 1024, "bf16"
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    w = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    ws = (torch.randint(1, 5, (N, K // G), device="cuda", generator=gen) * 2.0 ** -6).to(DT[T])
    rows = torch.cat([torch.arange(8), torch.arange(299_996, 300_000), torch.arange(N - 20, N)])
    part, spart = w[rows.cuda()].cpu().numpy(), ws[rows.cuda()].cpu()
    W, P = _mats(part, spart, None, G)
    for M in (1, 11, 20, 100):
        x = gen_x(M, K, T, seed=M, scale=0.1)
        y = ql.qlin_gemv_w4(x.cuda(), w, ws)[:, rows.cuda()]
        want, S, Q = ref.product(f64(x), W.T, P.T)
        close(y, want, ref.rounded_tolerance(want, ref.sum_tolerance(S, Q, K, T, M <= 16), T), f"M={M}")
    for M in (2, 70):
        dy = torch.zeros((M, N), dtype=DT[T], device="cuda")
        vals = gen_x(M, len(rows), T, seed=M)
        dy[:, rows.cuda()] = vals.cuda()
        dx = ql.qlin_gemv_w4_bwd(dy, w, ws)
        want, S, Q = ref.product(f64(vals), W, P)
        close(dx, want, ref.rounded_tolerance(want, ref.sum_tolerance(S, Q, len(rows), T, False), T), f"dx M={M}")
