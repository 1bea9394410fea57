"""Results and workspaces that the 8-bit and expert calls allocate for themselves, on a stream of the caller's: the
memory belongs to that stream, so work of the current one neither overwrites it nor is overwritten."""
import pytest
import torch

from gpu_util import dev, dev_bf16, lib, need_gpu

pytestmark = pytest.mark.gpu

M, N, K = 4, 1536, 1024


@pytest.fixture(scope="module")
def calls():
    need_gpu()
    ql = lib()
    from skinny_gemm_qlin_amd.inputs import gen_fp8, gen_fp8_blk, gen_fp8_w8a8, gen_int8, gen_moe, gen_moe_ffn
    i8, f8, b8 = gen_int8(M, N, K, seed=0), gen_fp8(M, N, K, seed=0), gen_fp8_blk(M, N, K, seed=0)
    c8, moe, ffn = gen_fp8_w8a8(M, N, K, seed=0), gen_moe(M, 8, N, 512, 2, seed=0), gen_moe_ffn(M, 8, 1024, 512, 2, seed=0)
    x, w, ws = dev_bf16(i8["x"]), dev(i8["w"]), dev(i8["ws"])
    xq, xs = ql.qlin_act_quant_i8(x)
    fx, fw, fs = dev_bf16(f8["x"]), dev(f8["w"]), dev(f8["ws"])
    bx, bw, bs = dev_bf16(b8["x"]), dev(b8["w"]), dev(b8["ws"])
    cx, cw, cs = dev_bf16(c8["x"]), dev(c8["w"]), dev(c8["ws"])
    cq, cqs = ql.qlin_act_quant_fp8(cx)
    mo = (dev_bf16(moe["x"]), dev(moe["w"]), dev(moe["s"]), dev(moe["ids"]), dev(moe["gw"]))
    ff = (dev_bf16(ffn["x"]), dev_bf16(ffn["wr"]), dev(ffn["w13"]), dev(ffn["s13"]), dev(ffn["w2"]), dev(ffn["s2"]), 2)
    one = bx[:1].contiguous()
    torch.cuda.synchronize()
    # name -> call(stream, outputs): a tuple of all outputs
    return {
        "act_quant_i8": lambda **k: ql.qlin_act_quant_i8(x, **k),
        "gemv_i8": lambda **k: (ql.qlin_gemv_i8(xq, xs, w, ws, **k),),
        "linear_i8": lambda **k: ql.qlin_linear_i8(x, w, ws, **k),
        "gemv_fp8": lambda **k: (ql.qlin_gemv_fp8(fx, fw, fs, **k),),
        "act_quant_fp8": lambda **k: ql.qlin_act_quant_fp8(cx, **k),
        "gemv_fp8_w8a8": lambda **k: (ql.qlin_gemv_fp8_w8a8(cq, cqs, cw, cs, **k),),
        "gemv_fp8_blk": lambda **k: ql.qlin_gemv_fp8_blk(bx, bw, bs, **k),
        "gemv_fp8_blk one token": lambda **k: ql.qlin_gemv_fp8_blk(one, bw, bs, export=False, **k)[:1],
        "gemv_fp8_blk_ex": lambda **k: ql.qlin_gemv_fp8_blk_ex(bx, bw, bs.repeat_interleave(2, 0), 64, 128, **k),
        "moe_mxfp4": lambda **k: (ql.qlin_moe_mxfp4(*mo, **k),),
        "moe_ffn_mxfp4": lambda **k: ql.qlin_moe_ffn_mxfp4(*ff, **k),
    }


NAMES = ("act_quant_i8", "gemv_i8", "linear_i8", "gemv_fp8", "act_quant_fp8", "gemv_fp8_w8a8", "gemv_fp8_blk",
         "gemv_fp8_blk one token", "gemv_fp8_blk_ex", "moe_mxfp4", "moe_ffn_mxfp4")


def _same(got, want):
    return all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_memory_of_the_call_is_the_streams(calls, name, raw):
    """Right results by either kind of handle, and what is dropped is not handed out on the current stream."""
    want = [t.clone() for t in calls[name]()]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = calls[name](stream=st.cuda_stream if raw else st)
    torch.cuda.synchronize()
    assert _same(got, want)
    blocks = [(t.data_ptr(), t.numel() * t.element_size()) for t in got]
    del got
    for ptr, size in blocks:
        fresh = [torch.empty((size,), dtype=torch.uint8, device="cuda") for _ in range(50)]
        assert all(t.data_ptr() != ptr for t in fresh)


@pytest.mark.parametrize("name", ["moe_mxfp4", "moe_ffn_mxfp4"])
def test_workspace_is_not_taken_away(calls, name):
    """The call waits on its stream behind other work; blocks of every size near the dropped workspace's are filled
    on the current stream in the meantime."""
    want = [t.clone() for t in calls[name]()]
    held = torch.empty_like(want[0])
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        a = torch.ones((4096, 4096), device="cuda")
        for _ in range(12):
            a = torch.mm(a, a)
    calls[name](stream=st, y=held)
    junk = [torch.full((size,), 255, dtype=torch.uint8, device="cuda")
            for size in (4096, 16384, 49152, 65536, 98304, 131072) for _ in range(20)]
    st.synchronize()
    assert _same([held], want[:1])
    del junk, a


def test_the_default_stream_by_its_handle(calls):
    """Handle 0 from within another stream."""
    want = [t.clone() for t in calls["linear_i8"]()]
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = calls["linear_i8"](stream=0)
    torch.cuda.synchronize()
    assert _same(got, want)
