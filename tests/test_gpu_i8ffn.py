"""The INT8 feed-forward operators against their 64-bit definition: sizes, types, routings."""
import numpy as np
import pytest
import torch

from gpu_util import lib, need_gpu
from i8ffn_util import check_glu, check_moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ql():
    need_gpu()
    return lib()


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("M,I,K", [(1, 1, 16), (1, 33, 48), (1, 512, 1024), (2, 100, 144), (3, 65, 2064), (5, 257, 4096),
                                   (8, 64, 5120), (16, 130, 1040), (17, 96, 256), (31, 100, 400), (64, 64, 128),
                                   (65, 129, 272), (130, 200, 1024), (300, 300, 528)])
def test_glu_sizes(ql, M, I, K, dt):
    check_glu(ql, M, I, K, dt, seed=M + I)


@pytest.mark.parametrize("K", [16, 128, 144, 384, 512, 640, 1040])
@pytest.mark.parametrize("M,I", [(40, 8200), (70, 4100), (120, 8300), (130, 8200), (700, 5600), (1030, 6700)])
def test_glu_tiles(ql, M, I, K):
    """Widths that take every tile of the matrix kernel, with one to nine steps of K."""
    check_glu(ql, M, I, K, "bf16" if K % 128 else "fp16", seed=K)


@pytest.mark.parametrize("M", [1, 4, 16, 40])
def test_glu_variants(ql, M):
    check_glu(ql, M, 50, 320, "bf16", kind=1, seed=1)
    check_glu(ql, M, 50, 320, "fp16", kind=1, seed=2, pad=32)
    check_glu(ql, M, 50, 320, "bf16", seed=3, one_scale=True, pad=16)


@pytest.mark.parametrize("M,I,K", [(1, 40, 65536), (1, 24, 131072), (3, 20, 40000), (16, 16, 65536), (20, 16, 131072)])
def test_glu_long_rows(ql, M, I, K):
    check_glu(ql, M, I, K, "bf16", seed=K)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("M,E,topk,H,I", [
    (1, 1, 1, 16, 16), (1, 8, 2, 256, 64), (1, 64, 6, 512, 128), (2, 4, 4, 144, 48), (3, 128, 8, 272, 80),
    (5, 3, 2, 1040, 1040), (8, 64, 6, 512, 128), (13, 40, 5, 336, 112), (16, 16, 16, 128, 32), (16, 8, 2, 256, 512),
    (16, 1, 1, 512, 64), (17, 200, 8, 128, 64), (40, 8, 2, 256, 96), (64, 32, 4, 272, 96), (70, 1024, 8, 64, 32),
    (200, 4, 2, 256, 128), (300, 16, 4, 144, 144), (1, 1024, 16, 64, 32), (16, 1024, 16, 48, 32), (5, 700, 16, 4096, 16),
    (16, 130, 3, 528, 1040)])
def test_moe_sizes(ql, M, E, topk, H, I, dt):
    check_moe(ql, M, E, topk, H, I, dt, seed=M + E)


@pytest.mark.parametrize("M", [1, 7, 16, 33, 90])
def test_moe_variants(ql, M):
    check_moe(ql, M, 12, 3, 256, 96, "bf16", mode=1, seed=M)
    check_moe(ql, M, 12, 3, 256, 96, "fp16", kind=1, mode=1, seed=M + 1, pad=48)
    check_moe(ql, M, 12, 3, 256, 96, "bf16", seed=M + 2, given=True, pad=16)
    check_moe(ql, M, 5, 7, 80, 64, "fp16", kind=1, seed=M + 3, given=True)  # more slots than experts


@pytest.mark.parametrize("K", [16, 128, 144, 384, 640])
@pytest.mark.parametrize("M,E,topk", [(40, 8, 2), (90, 8, 2), (90, 2, 2)])
def test_moe_tiles(ql, M, E, topk, K):
    """Tiles of 32, 64 and 128 rows, with one to five steps of either reduction."""
    check_moe(ql, M, E, topk, K, 208, "bf16", seed=K)
    check_moe(ql, M, E, topk, 208, K, "fp16", seed=K)


@pytest.mark.parametrize("M,E,topk,H,I", [(1, 2, 1, 40000, 32), (2, 2, 2, 48, 65536), (20, 2, 1, 40000, 32),
                                          (3, 1, 1, 131072, 16), (2, 2, 2, 16, 131072)])
def test_moe_long_rows(ql, M, E, topk, H, I):
    check_moe(ql, M, E, topk, H, I, "bf16", seed=H)


def test_experts_only_one_is_asked_for(ql):
    """Every token goes to one expert: the largest count of one and none of all others."""
    from i8ffn_util import cuda, f64, gen_layer, gen_x, check
    from oracle import i8ffn
    for M in (1, 9, 16, 50, 150):
        x, (w13, s13, w2, s2) = gen_x(M, 256, "bf16", M), gen_layer(6, 256, 64, M)
        ids = np.full((M, 1), 4, dtype=np.int32)
        gw = np.ones((M, 1), dtype=np.float32)
        y, _, _ = ql.qlin_moe_ffn_i8(cuda(x), w13.cuda(), s13.cuda(), w2.cuda(), s2.cuda(),
                                     ids=torch.from_numpy(ids).cuda(), gw=torch.from_numpy(gw).cuda())
        want, tol = i8ffn.layer(f64(x), ids, gw, w13.numpy(), s13.numpy(), w2.numpy(), s2.numpy(), 0, "bf16")
        check(y, want, tol, f"one expert, {M} tokens")
