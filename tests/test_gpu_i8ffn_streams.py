"""The INT8 feed-forward calls on streams of the caller's, in graphs, from several threads, and together as a model
uses them."""
import threading

import pytest
import torch

from gpu_util import lib, need_gpu
from i8ffn_util import DT, check, f64, gen_codes, gen_layer, gen_logits, gen_scales, gen_x
from oracle import i8ffn

pytestmark = pytest.mark.gpu

I, K, E, TOPK, F = 500, 1024, 8, 2, 208


@pytest.fixture(scope="module")
def ql():
    need_gpu()
    return lib()


@pytest.fixture(scope="module")
def weights():
    return ((gen_codes((2 * I, K), 1).cuda(), gen_scales((2 * I,), K, 2).cuda()),
            tuple(t.cuda() for t in gen_layer(E, K, F, 3)))


def data(M, seed=5):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(-1, E, (M, TOPK), generator=g, dtype=torch.int32)
    return gen_x(M, K, "bf16", seed).cuda(), gen_logits(M, E, seed + 1).cuda(), ids.cuda(), torch.rand((M, TOPK), generator=g).cuda()


def calls(ql, weights, d):
    """name -> (call, the names of what it returns, in order)"""
    x, lg, ids, gw = d
    front, layer = weights
    return {"glu": (lambda **k: ql.qlin_glu_i8(x, *front, **k), ("y", "xq", "xs")),
            "moe": (lambda **k: ql.qlin_moe_ffn_i8(x, *layer, logits=lg, topk=TOPK, **k), ("y", "ids", "gw")),
            "given": (lambda **k: ql.qlin_moe_ffn_i8(x, *layer, ids=ids, gw=gw, **k)[:1], ("y",))}


NAMES, SIZES = ("glu", "moe", "given"), (1, 8, 40)


def same(got, want):
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def busy(stream, times=12):
    """Some milliseconds of work on `stream`."""
    with torch.cuda.stream(stream):
        a = torch.ones((4096, 4096), device="cuda")
        for _ in range(times):
            a = torch.mm(a, a)
    return a


def workspace(ql, M):
    return torch.empty((ql.qlin_moe_ffn_i8_workspace_bytes(M, K, F, TOPK, E),), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("M", SIZES)
@pytest.mark.parametrize("name", NAMES)
def test_memory_of_the_call_is_the_streams(ql, weights, name, M):
    """What the call allocated and dropped is not handed out on the current stream."""
    call, _ = calls(ql, weights, data(M))[name]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = call(stream=st)
    torch.cuda.synchronize()
    held = [(t.data_ptr(), t.shape, t.dtype) for t in got]
    del got
    for ptr, shape, dtype in held:
        fresh = [torch.empty(shape, dtype=dtype, device="cuda") for _ in range(50)]
        assert all(t.data_ptr() != ptr for t in fresh)


@pytest.mark.parametrize("M", SIZES)
@pytest.mark.parametrize("name", NAMES)
def test_later_work_of_the_current_stream(ql, weights, name, M):
    """Outputs that the caller holds are right although blocks of every size that the call dropped are taken and filled
    on the current stream while the call still waits on its own."""
    call, outs = calls(ql, weights, data(M))[name]
    want = [t.clone() for t in call()]
    held = {outs[0]: torch.empty_like(want[0])}
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    work = busy(st)
    call(stream=st, **held)
    junk = [torch.full(t.shape, 1, dtype=t.dtype, device="cuda") for t in want for _ in range(20)]
    junk += [workspace(ql, M).fill_(255) for _ in range(4)]
    st.synchronize()
    assert torch.equal(held[outs[0]], want[0])
    del work, junk


@pytest.mark.parametrize("M", SIZES)
@pytest.mark.parametrize("name", NAMES)
def test_earlier_work_of_the_current_stream(ql, weights, name, M):
    """Outputs and workspace of the call's own are right although blocks of their sizes are still to be filled by the
    current stream."""
    call, _ = calls(ql, weights, data(M))[name]
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    work = busy(torch.cuda.current_stream())
    junk = [torch.full(t.shape, 1, dtype=t.dtype, device="cuda") for t in want for _ in range(20)]
    junk += [workspace(ql, M).fill_(255) for _ in range(4)]
    del junk
    got = call(stream=st)
    torch.cuda.synchronize()
    same(got, want)
    del work


@pytest.mark.parametrize("M", SIZES)
@pytest.mark.parametrize("name", NAMES)
def test_raw_handles(ql, weights, name, M):
    """A raw handle, with buffers of the caller's, with some of them, and with none; the current stream's own."""
    call, outs = calls(ql, weights, data(M))[name]
    want = [t.clone() for t in call()]
    st = torch.cuda.Stream()
    bufs = {o: torch.empty_like(t) for o, t in zip(outs, want)}
    if name != "glu":
        bufs["workspace"] = workspace(ql, M)
    torch.cuda.synchronize()
    for given in (bufs, {}, *({k: v for k, v in bufs.items() if k != left_out} for left_out in bufs)):
        got = call(stream=st.cuda_stream, **given)
        st.synchronize()
        same(got, want)
        for t in bufs.values():
            t.fill_(1)
        torch.cuda.synchronize()
    same(call(stream=torch.cuda.current_stream().cuda_stream), want)


def feed(M, seeds):
    return [data(M, s) for s in seeds]


@pytest.mark.parametrize("M", (1, 4, 13, 16, 40, 300))
def test_graph(ql, weights, M):
    """Both calls and the given form, buffers of the caller's; new tokens and routings each replay, eager work between."""
    front, layer = weights
    x, lg, ids, gw = (t.clone() for t in data(M))
    xq, xs = torch.empty((M, K), dtype=torch.int8, device="cuda"), torch.empty((M,), device="cuda")
    y, z, v = (torch.empty((M, n), dtype=x.dtype, device="cuda") for n in (I, K, K))
    oi, og = torch.empty_like(ids), torch.empty_like(gw)
    work = workspace(ql, M)

    def step():
        ql.qlin_glu_i8(x, *front, xq=xq, xs=xs, y=y)
        ql.qlin_moe_ffn_i8(x, *layer, logits=lg, topk=TOPK, ids=oi, gw=og, y=z, workspace=work)
        ql.qlin_moe_ffn_i8(x, *layer, ids=ids, gw=gw, y=v, workspace=work)
        return xq, xs, y, oi, og, z, v

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for d in feed(M, (11, 12, 13, 14)):
        for a, b in zip((x, lg, ids, gw), d):
            a.copy_(b)
        for t in outs:
            t.fill_(1)
        work.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        same(got, step())
        torch.cuda.synchronize()


@pytest.mark.parametrize("M", (1, 13, 40))
def test_two_graphs_at_once(ql, weights, M):
    """Graphs whose calls allocate for themselves have workspaces of their own: replayed together on two streams."""
    _, layer = weights
    one, two = data(M, 21), data(M, 22)
    want = [ql.qlin_moe_ffn_i8(d[0], *layer, logits=d[1], topk=TOPK)[0].clone() for d in (one, two)]
    graphs = []
    for d in (one, two):
        ql.qlin_moe_ffn_i8(d[0], *layer, logits=d[1], topk=TOPK)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = [ql.qlin_moe_ffn_i8(d[0], *layer, logits=d[1], topk=TOPK)[0] for _ in range(4)]
        graphs.append((g, outs, torch.cuda.Stream()))
    for _ in range(10):
        for g, _, st in graphs:
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for (_, outs, _), w in zip(graphs, want):
            for t in outs:
                assert torch.equal(t, w)
                t.fill_(0)
        torch.cuda.synchronize()


@pytest.mark.parametrize("M", (1, 16, 40))
def test_threads(ql, weights, M):
    """Four threads, each on a stream of its own, all calls."""
    sets = feed(M, (31, 32, 33, 34))
    want = [[[t.clone() for t in c()] for c, _ in calls(ql, weights, d).values()] for d in sets]
    torch.cuda.synchronize()
    fails = []

    def run(d, w):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                for _ in range(8):
                    for (call, _), ref in zip(calls(ql, weights, d).values(), w):
                        got = call()
                        st.synchronize()
                        same(got, ref)
        except Exception as e:  # reported by the main thread
            fails.append(repr(e))

    threads = [threading.Thread(target=run, args=a) for a in zip(sets, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not fails, fails


@pytest.mark.parametrize("M", (1, 12, 48))
def test_a_block_with_a_shared_expert(ql, weights, M):
    """A router's product, the routed layer and, beside it on another stream, a shared expert (front and down
    projection) added to it, over several steps; each against the definition from what it was given."""
    front, (w13, s13, w2, s2) = weights
    down, sd = gen_codes((K, 512), 7).cuda(), gen_scales((K,), 512, 8).cuda()
    wide, sw = gen_codes((1024, K), 9).cuda(), gen_scales((1024,), K, 10).cuda()
    router = torch.randn((E, K), generator=torch.Generator().manual_seed(1)).cuda() / K ** 0.5
    x, side = data(M, 41)[0], torch.cuda.Stream()
    for _ in range(3):
        here = torch.cuda.current_stream()
        lg = torch.mm(x.float(), router.t())
        side.wait_stream(here)
        h, xq, xs = ql.qlin_glu_i8(x, wide, sw, stream=side)
        y, hq, hs = ql.qlin_linear_i8(h, down, sd, stream=side)
        z, ids, gw = ql.qlin_moe_ffn_i8(x, w13, s13, w2, s2, logits=lg, topk=TOPK)
        here.wait_stream(side)
        out = x + y + z
        torch.cuda.synchronize()
        q, s = i8ffn.quantise(f64(x))
        want, _, tol = i8ffn.front(q, s, wide.cpu().numpy(), sw.cpu().numpy(), 0, "bf16")
        check(h, want, tol, "shared expert's front")
        q, s = i8ffn.quantise(f64(h))
        want = (q @ f64(down).T) * s[:, None] * f64(sd)
        check(y, want, abs(want) * (2.0 ** -8 + 2.0 ** -20) + 1e-30, "shared expert's down")
        wids, wgw = i8ffn.route(lg.cpu().numpy(), TOPK, 0)
        assert (ids.cpu().numpy() == wids).all() and abs(f64(gw) - wgw).max() < 2.0 ** -18
        want, tol = i8ffn.layer(f64(x), wids, f64(gw), *(t.cpu().numpy() for t in (w13, s13, w2, s2)), 0, "bf16")
        check(z, want, tol, "routed")
        x = (out * torch.rsqrt(out.float().pow(2).mean(-1, keepdim=True))).to(DT["bf16"])


# ------------------------------------------------------------------ torch operators

@pytest.fixture(scope="module")
def ops():
    need_gpu()
    lib()
    import skinny_gemm_qlin_amd.torch_ops as t
    return t


@pytest.mark.parametrize("M", (1, 20))
def test_operator_checks(ops, ql, weights, M):
    front, layer = weights
    x, lg, ids, gw = data(M)
    before = dict(ops.hits)
    y = torch.ops.qlin.glu_i8(x, *front, 1)
    z = torch.ops.qlin.moe_ffn_i8(x, *layer, lg, TOPK, 1, 1)
    v = torch.ops.qlin.moe_ffn_i8_given(x, *layer, ids, gw, 1)
    for name in ("glu_i8", "moe_ffn_i8", "moe_ffn_i8_given"):
        assert ops.hits[name] == before.get(name, 0) + 1
    assert torch.equal(y, ql.qlin_glu_i8(x, *front, act=1)[0])
    same(z, ql.qlin_moe_ffn_i8(x, *layer, logits=lg, topk=TOPK, route=1, act=1))
    assert torch.equal(v, ql.qlin_moe_ffn_i8(x, *layer, ids=ids, gw=gw, act=1)[0])
    torch.library.opcheck(torch.ops.qlin.glu_i8.default, (x, *front, 1))
    torch.library.opcheck(torch.ops.qlin.moe_ffn_i8.default, (x, *layer, lg, TOPK, 1, 0))
    torch.library.opcheck(torch.ops.qlin.moe_ffn_i8_given.default, (x, *layer, ids, gw))


@pytest.mark.parametrize("M", (1, 20))
def test_compiled(ops, weights, M):
    front, layer = weights
    x, lg, _, _ = data(M)

    def block(x, lg):
        return x + torch.ops.qlin.moe_ffn_i8(x, *layer, lg, TOPK)[0], torch.ops.qlin.glu_i8(x, *front)

    same(torch.compile(block, backend="aot_eager", fullgraph=True)(x, lg), block(x, lg))
