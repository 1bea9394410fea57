"""The INT8 feed-forward calls at the largest number of tokens, and the layer at the largest number of pairs."""
import numpy as np
import pytest
import torch

from gpu_util import lib, need_gpu
from i8ffn_util import check, check_glu, f64, gen_layer, gen_x
from oracle import i8ffn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ql():
    need_gpu()
    return lib()


def test_front_of_16384_tokens(ql):
    check_glu(ql, 16384, 37, 48, "bf16", seed=1)


@pytest.mark.parametrize("E,spread", [(1024, "even"), (1024, "one"), (3, "even"), (1, "one")])
def test_layer_of_16384_tokens_and_16_slots(ql, E, spread):
    """262144 pairs: over all experts, or all but a few of them to the last one; some slots without an expert."""
    M, topk, H, I = 16384, 16, 16, 32
    rng = np.random.default_rng(E)
    ids = rng.integers(0, E, (M, topk)).astype(np.int32)
    if spread == "one":
        ids[rng.random((M, topk)) < 0.99] = E - 1
    ids[rng.random((M, topk)) < 0.05] = -1
    gw = rng.uniform(0.0, 0.2, (M, topk)).astype(np.float32)
    x, (w13, s13, w2, s2) = gen_x(M, H, "bf16", 1), gen_layer(E, H, I, 2)
    y, _, _ = ql.qlin_moe_ffn_i8(x.cuda(), w13.cuda(), s13.cuda(), w2.cuda(), s2.cuda(), ids=torch.from_numpy(ids).cuda(),
                                 gw=torch.from_numpy(gw).cuda())
    want, tol = i8ffn.layer(f64(x), ids, gw, w13.numpy(), s13.numpy(), w2.numpy(), s2.numpy(), 0, "bf16")
    check(y, want, tol, f"{E} experts, {spread}")
