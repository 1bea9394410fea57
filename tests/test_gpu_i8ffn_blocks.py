"""The INT8 expert layer for up to 16 tokens where a workgroup of the down projection has several blocks of row groups,
and where LDS does not hold the codes of all pairs: against the definition, and bit for bit against other batches."""
import numpy as np
import pytest
import torch

from gpu_util import lib, need_gpu
from i8ffn_block_cases import CASES
from i8ffn_util import check, check_moe, cuda, f64, gen_layer, gen_logits, gen_x
from oracle import i8ffn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ql():
    need_gpu()
    return lib()


def bits(t):
    return t.contiguous().view(torch.int16)


def given(M, E, topk, seed, hole=0.3):
    """Experts and weights of the caller's: slots without an expert, the same one twice, a token without any."""
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, E, (M, topk)).astype(np.int32)
    ids[rng.random((M, topk)) < hole] = -1
    if M > 1:
        ids[M // 2] = E
    return torch.from_numpy(ids), torch.from_numpy(rng.standard_normal((M, topk)).astype(np.float32))


@pytest.mark.parametrize("M,E,topk,H,I,whole", CASES)
def test_from_logits_and_given(ql, M, E, topk, H, I, whole):
    """All slots live (as many as there are experts), and with holes."""
    check_moe(ql, M, E, min(topk, E), H, I, "bf16", seed=H + I)
    check_moe(ql, M, E, topk, H, I, "fp16", kind=1, seed=H + M, given=True)


@pytest.mark.parametrize("M,E,topk,H,I,whole", CASES)
def test_every_slot_live(ql, M, E, topk, H, I, whole):
    """Twice into buffers and a workspace that hold junk: the definition, and the same bits."""
    x, (w13, s13, w2, s2) = gen_x(M, H, "bf16", M), gen_layer(E, H, I, E)
    ids, gw = given(M, E, topk, H, hole=0.0)
    ids[M // 2] = E - 1
    dev = [cuda(x), w13.cuda(), s13.cuda(), w2.cuda(), s2.cuda()]
    work = torch.empty((ql.qlin_moe_ffn_i8_workspace_bytes(M, H, I, topk, E),), dtype=torch.uint8, device="cuda")
    first = None
    for junk in (255, 0):
        work.fill_(junk)
        y = torch.full((M + 1, H + 3), float("nan"), dtype=x.dtype, device="cuda")
        ql.qlin_moe_ffn_i8(*dev, ids=ids.cuda(), gw=gw.cuda(), y=y[:M, :H], workspace=work)
        assert torch.isnan(y[M:]).all() and torch.isnan(y[:, H:]).all()
        if first is not None:
            assert torch.equal(bits(y[:M, :H]), first)
        first = bits(y[:M, :H])
    want, tol = i8ffn.layer(f64(x), ids.numpy(), gw.numpy(), w13.numpy(), s13.numpy(), w2.numpy(), s2.numpy(), 0, "bf16")
    check(y[:M, :H], want, tol, f"{M} x {E} top {topk} {H} x {I}")


@pytest.mark.parametrize("M,E,topk,H,I,whole", CASES)
def test_a_token_does_not_see_its_batch(ql, M, E, topk, H, I, whole):
    """Each of the tokens alone, half of them, and among 40: the same bits."""
    x, layer = gen_x(40, H, "bf16", 7).cuda(), [t.cuda() for t in gen_layer(E, H, I, 8)]
    ids, gw = (t.cuda() for t in given(40, E, topk, 9))
    every = ql.qlin_moe_ffn_i8(x, *layer, ids=ids, gw=gw)[0]

    def part(a, b):
        return ql.qlin_moe_ffn_i8(x[a:b], *layer, ids=ids[a:b].contiguous(), gw=gw[a:b].contiguous())[0]

    assert torch.equal(bits(part(0, M)), bits(every[:M]))
    assert torch.equal(bits(part(0, (M + 1) // 2)), bits(every[:(M + 1) // 2]))
    for t in {0, M // 2, M - 1}:
        assert torch.equal(bits(part(t, t + 1)), bits(every[t:t + 1]))


@pytest.mark.parametrize("M,E,topk,H,I,whole", [c for c in CASES if c[0] == 16])
def test_graph_of_several_blocks(ql, M, E, topk, H, I, whole):
    """Captured once, replayed on other tokens and routings, eager work between."""
    layer = [t.cuda() for t in gen_layer(E, H, I, 3)]
    x, lg, k = gen_x(M, H, "bf16", 1).cuda(), gen_logits(M, E, 2).cuda(), min(topk, E)
    ids, gw = (t.cuda() for t in given(M, E, topk, 4))
    oi, og = torch.empty((M, k), dtype=torch.int32, device="cuda"), torch.empty((M, k), device="cuda")
    y, z = torch.empty_like(x), torch.empty_like(x)
    work = torch.empty((ql.qlin_moe_ffn_i8_workspace_bytes(M, H, I, topk, E),), dtype=torch.uint8, device="cuda")

    def step():
        ql.qlin_moe_ffn_i8(x, *layer, logits=lg, topk=k, ids=oi, gw=og, y=y, workspace=work)
        ql.qlin_moe_ffn_i8(x, *layer, ids=ids, gw=gw, y=z, workspace=work)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in (11, 12, 13):
        x.copy_(gen_x(M, H, "bf16", seed))
        lg.copy_(gen_logits(M, E, seed + 1))
        for a, b in zip((ids, gw), given(M, E, topk, seed + 2)):
            a.copy_(b)
        y.fill_(1), z.fill_(1), work.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        got = y.clone(), z.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(bits(got[0]), bits(y)) and torch.equal(bits(got[1]), bits(z))
