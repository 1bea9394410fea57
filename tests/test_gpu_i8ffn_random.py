"""The INT8 feed-forward operators at shapes drawn over their ranges."""
import random

import pytest

from gpu_util import lib, need_gpu
from i8ffn_util import check_glu, check_moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ql():
    need_gpu()
    return lib()


def _tokens(r):
    return r.choice((1, r.randint(2, 16), r.randint(17, 64), r.randint(65, 400)))


@pytest.mark.parametrize("seed", range(30))
def test_front(ql, seed):
    r = random.Random(seed)
    M, K = _tokens(r), 16 * r.randint(1, 200)
    check_glu(ql, M, r.randint(1, 600), K, r.choice(("bf16", "fp16")), kind=r.randint(0, 1), seed=seed,
              pad=8 * r.randint(0, 5), one_scale=r.random() < 0.3)


@pytest.mark.parametrize("seed", range(30))
def test_layer(ql, seed):
    r = random.Random(1000 + seed)
    M, E = _tokens(r), r.choice((1, 2, r.randint(3, 16), r.randint(17, 80), r.randint(81, 300)))
    H, I = 16 * r.randint(1, 80), 16 * r.randint(1, 40)
    if E > 80:
        H, I = min(H, 512), min(I, 256)
    check_moe(ql, M, E, r.randint(1, min(E, 16)), H, I, r.choice(("bf16", "fp16")), kind=r.randint(0, 1),
              mode=r.randint(0, 1), seed=seed, pad=8 * r.randint(0, 5), given=r.random() < 0.3)
