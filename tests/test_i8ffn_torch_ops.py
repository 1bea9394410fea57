"""The INT8 feed-forward custom operators: shapes and types without a GPU."""
import pytest
import torch

import skinny_gemm_qlin_amd.torch_ops  # noqa: F401


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_fake_results(dt):
    with torch.device("meta"):
        x = torch.empty((5, 64), dtype=dt)
        y = torch.ops.qlin.glu_i8(x, torch.empty((14, 64), dtype=torch.int8), torch.empty((14,)))
        assert y.shape == (5, 7) and y.dtype is dt
        layer = (torch.empty((4, 32, 64), dtype=torch.int8), torch.empty((4, 32)),
                 torch.empty((4, 64, 16), dtype=torch.int8), torch.empty((4, 64)))
        y, ids, gw = torch.ops.qlin.moe_ffn_i8(x, *layer, torch.empty((5, 4)), 3)
        assert y.shape == (5, 64) and y.dtype is dt
        assert ids.shape == gw.shape == (5, 3) and ids.dtype is torch.int32 and gw.dtype is torch.float32
        y = torch.ops.qlin.moe_ffn_i8_given(x, *layer, torch.empty((5, 2), dtype=torch.int32), torch.empty((5, 2)))
        assert y.shape == (5, 64) and y.dtype is dt
