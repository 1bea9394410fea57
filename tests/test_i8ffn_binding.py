"""Operands of the INT8 feed-forward calls that the binding refuses, by name (no GPU)."""
import numpy as np
import pytest
import torch

import skinny_gemm_qlin_amd as ql

X = torch.zeros((2, 64), dtype=torch.bfloat16)
W = torch.zeros((8, 64), dtype=torch.int8)
S = torch.zeros((8,), dtype=torch.float32)
E13, S13 = torch.zeros((3, 32, 64), dtype=torch.int8), torch.zeros((3, 32))
E2, S2 = torch.zeros((3, 64, 16), dtype=torch.int8), torch.zeros((3, 64))


@pytest.mark.parametrize("bad", [None, 3, "x", [1.0], np.zeros((2, 64), np.float32)])
def test_first_operand_that_is_no_tensor(bad):
    with pytest.raises(TypeError, match="x: expected a torch.Tensor"):
        ql.qlin_glu_i8(bad, W, S)
    with pytest.raises(TypeError, match="x: expected a torch.Tensor"):
        ql.qlin_moe_ffn_i8(bad, E13, S13, E2, S2, logits=torch.zeros((2, 3)), topk=1)


@pytest.mark.parametrize("call", [lambda x: ql.qlin_glu_i8(x, W, S),
                                  lambda x: ql.qlin_moe_ffn_i8(x, E13, S13, E2, S2, logits=torch.zeros((2, 3)), topk=1)])
def test_host_tensors_and_types(call):
    with pytest.raises(ValueError, match="x: must be a device tensor"):
        call(X)
    with pytest.raises(TypeError, match="x: dtype torch.float32"):
        call(X.float())
    with pytest.raises(ValueError, match="x: "):
        call(X[0])


def test_expert_pitch():
    assert ql._expert_pitch(E13) == 64
    pad = torch.zeros((3, 32, 80), dtype=torch.int8)
    assert ql._expert_pitch(pad[:, :, :64]) == 80
    assert ql._expert_pitch(pad[:, :16, :64]) is None          # experts not one behind the other
    assert ql._expert_pitch(pad[:1, :16, :64]) == 80           # a single one has nothing to be behind
    assert ql._expert_pitch(E13.transpose(1, 2)) is None
    assert ql._expert_pitch(torch.zeros((2, 1, 64), dtype=torch.int8)) == 64
    assert ql._expert_pitch(torch.zeros((1, 1, 64), dtype=torch.int8)) == 64
