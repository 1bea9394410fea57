"""A dense feed-forward block as the INT8 layer of one expert: what an fp16 block takes in place of qlin_glu_i8 and
qlin_linear_i8, whose activations are bf16."""
import numpy as np
import pytest
import torch

from gpu_util import lib, need_gpu
from i8ffn_util import check, f64, gen_layer, gen_x
from oracle import i8ffn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ql():
    need_gpu()
    return lib()


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("M,H,I", [(1, 1024, 512), (7, 272, 1040), (16, 512, 208), (40, 528, 96), (200, 144, 272), (1040, 128, 256)])
def test_one_expert_is_a_dense_block(ql, M, H, I, kind, dt):
    """The layer's row is the down projection of the front's own output, rounded once."""
    x, (w13, s13, w2, s2) = gen_x(M, H, dt, M + I).cuda(), (t.cuda() for t in gen_layer(1, H, I, M))
    ids, gw = torch.zeros((M, 1), dtype=torch.int32, device="cuda"), torch.ones((M, 1), device="cuda")
    y = ql.qlin_moe_ffn_i8(x, w13, s13, w2, s2, ids=ids, gw=gw, act=kind)[0]
    h = ql.qlin_glu_i8(x, w13[0], s13[0], act=kind)[0]
    q, s = i8ffn.quantise(f64(h))
    want = (q @ f64(w2[0]).T) * s[:, None] * f64(s2[0])
    # the conversion of the whole-number sum and two products, 2^-24 each; a weight of one adds nothing; one rounding of y
    tol = np.abs(want) * (i8ffn.EPS16[dt] * (1 + 2.0 ** -20) + 3.01 * 2.0 ** -24) + i8ffn.TINY16[dt]
    assert y.dtype == x.dtype
    check(y, want, tol, f"dense block {M} x {H} x {I} {dt}")
