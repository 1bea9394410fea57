"""Sizes that the INT8 expert layer refuses are refused before anything is allocated for them."""
import pytest
import torch

from gpu_util import lib, need_gpu
from i8ffn_util import gen_layer, gen_logits, gen_x
from skinny_gemm_qlin_amd._lib import QlinError

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ql():
    need_gpu()
    return lib()


@pytest.mark.parametrize("topk", [-1, 0, 3, 17, 1 << 20, 1 << 40])
@pytest.mark.parametrize("held", [False, True])
def test_topk_outside_its_range(ql, topk, held):
    """Two experts: the status of a size outside the range, whatever the caller brings along; no memory is taken that
    grows with it."""
    layer = [t.cuda() for t in gen_layer(2, 64, 16, 1)]
    x, lg = gen_x(3, 64, "bf16", 1).cuda(), gen_logits(3, 2, 2).cuda()
    bufs = {}
    if held:
        bufs = dict(y=torch.empty_like(x), workspace=torch.empty((1 << 16,), dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    with pytest.raises(QlinError) as e:
        ql.qlin_moe_ffn_i8(x, *layer, logits=lg, topk=topk, **bufs)
    assert e.value.status == -2
    assert torch.cuda.max_memory_allocated() - before <= 1 << 16
    y, ids, _ = ql.qlin_moe_ffn_i8(x, *layer, logits=lg, topk=2, **bufs)
    assert torch.isfinite(y).all() and ids.shape == (3, 2)
