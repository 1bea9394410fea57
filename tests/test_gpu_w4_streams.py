"""Results, workspaces and intermediates that the 4-bit weight calls allocate for themselves, on a stream of the
caller's: the memory belongs to that stream, so work of the current one neither overwrites it nor is overwritten."""
import pytest
import torch

from gpu_util import lib, need_gpu
from w4_util import DT, dev_w, gen_w4, gen_x

pytestmark = pytest.mark.gpu

M, I, K = 40, 1000, 1024


@pytest.fixture(scope="module")
def ql():
    need_gpu()
    return lib()


@pytest.fixture(scope="module")
def layer():
    w, ws, wz = gen_w4(2 * I, K, 64, "bf16", True, seed=1)
    return dev_w(w, ws, wz)


@pytest.fixture(scope="module")
def data():
    x, dy, dgu = gen_x(M, K, "bf16", 1).cuda(), gen_x(M, I, "bf16", 2).cuda(), gen_x(M, 2 * I, "bf16", 3).cuda()
    return x, dy, dgu


def _calls(ql, layer, data):
    """name -> (call, the names of what it returns, in order)"""
    x, dy, big = data
    gu = big * 0.5
    return {"gemv": (lambda **k: (ql.qlin_gemv_w4(x, *layer, **k),), ("y",)),
            "gemv_bwd": (lambda **k: (ql.qlin_gemv_w4_bwd(big, *layer, **k),), ("dx",)),
            "glu": (lambda **k: (ql.qlin_glu_w4(x, *layer, **k),), ("y",)),
            "glu_bwd kept": (lambda **k: ql.qlin_glu_w4_bwd(dy, *layer, gu=gu, **k), ("dx", "dgu")),
            "glu_bwd recomputed": (lambda **k: ql.qlin_glu_w4_bwd(dy, *layer, x=x, **k), ("dx", "dgu"))}


NAMES = ("gemv", "gemv_bwd", "glu", "glu_bwd kept", "glu_bwd recomputed")


def _busy(stream, times=12):
    """Some milliseconds of work on `stream`."""
    with torch.cuda.stream(stream):
        a = torch.ones((4096, 4096), device="cuda")
        for _ in range(times):
            a = torch.mm(a, a)
    return a


@pytest.mark.parametrize("name", NAMES)
def test_memory_of_the_call_is_the_streams(ql, layer, data, name):
    """What the call allocated and dropped is not handed out on the current stream."""
    call, outs = _calls(ql, layer, data)[name]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = call(stream=st)
    torch.cuda.synchronize()
    shapes = [(t.data_ptr(), t.shape[0], t.stride(0)) for t in got]
    del got
    for ptr, rows, pitch in shapes:
        fresh = [torch.empty((rows, pitch), dtype=DT["bf16"], device="cuda") for _ in range(50)]
        assert all(t.data_ptr() != ptr for t in fresh)


@pytest.mark.parametrize("name", NAMES)
def test_later_work_of_the_current_stream(ql, layer, data, name):
    """Outputs that the caller holds are right although blocks of every size that the call dropped are taken and
    filled on the current stream while the call still waits on its own."""
    call, outs = _calls(ql, layer, data)[name]
    want = [t.clone() for t in call()]
    held = torch.empty_like(want[0])
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    busy = _busy(st)
    call(stream=st, **{outs[0]: held})
    junk = [torch.full((M, 2 * I), float("nan"), dtype=DT["bf16"], device="cuda") for _ in range(20)]
    junk += [torch.full((ql.qlin_gemv_w4_bwd_workspace_bytes(M, 2 * I, K) // 4,), float("nan"), device="cuda")
             for _ in range(4)]
    st.synchronize()
    assert torch.equal(held, want[0])
    del busy, junk


@pytest.mark.parametrize("name", NAMES)
def test_earlier_work_of_the_current_stream(ql, layer, data, name):
    """Outputs of the call's own are right although a block of their size is still to be filled by the current stream."""
    call, outs = _calls(ql, layer, data)[name]
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    busy = _busy(torch.cuda.current_stream())
    for t in want:  # blocks that go back to the current stream's memory with a fill still queued
        junk = [torch.full((t.shape[0], (t.shape[1] + 7) // 8 * 8), float("nan"), dtype=t.dtype, device="cuda")
                for _ in range(20)]
        del junk
    got = call(stream=st)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    del busy


@pytest.mark.parametrize("name", NAMES)
def test_raw_handles(ql, layer, data, name):
    """A raw handle comes with every buffer, unless it is the current stream's own."""
    call, outs = _calls(ql, layer, data)[name]
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    bufs = {o: torch.empty_like(t) for o, t in zip(outs, want)}
    if "dgu" in bufs:
        bufs["dgu"] = torch.empty((M, 2 * I), dtype=DT["bf16"], device="cuda")
    if "bwd" in name:
        need = ql.qlin_gemv_w4_bwd_workspace_bytes(M, 2 * I, K)
        assert need > 0
        bufs["workspace"] = torch.empty((need,), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for left_out in bufs:
        with pytest.raises(ValueError, match=f"raw stream.*{left_out}"):
            call(stream=st.cuda_stream, **{k: v for k, v in bufs.items() if k != left_out})
    got = call(stream=st.cuda_stream, **bufs)
    st.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    got = call(stream=torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_in_a_graph(ql, layer, data):
    """Forked inside a captured graph: outputs, intermediate and workspace of the calls' own, replayed."""
    x, dy, _ = data
    xs = x.clone()

    def step(st):
        here = torch.cuda.current_stream()
        st.wait_stream(here)
        gu = torch.empty((M, 2 * I), dtype=DT["bf16"], device="cuda")
        y = ql.qlin_glu_w4(xs, *layer, gu=gu, stream=st)
        dx, _ = ql.qlin_glu_w4_bwd(dy, *layer, gu=gu, stream=st)
        here.wait_stream(st)
        return y.clone(), dx.clone()

    side = torch.cuda.Stream()
    step(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step(side)
    for seed in (5, 6, 7):
        xs.copy_(gen_x(M, K, "bf16", seed))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        for a, b in zip(got, step(side)):
            assert torch.equal(a, b)
        torch.cuda.synchronize()
