"""Operands of the 4-bit weight calls that are no tensors: refused by name, like everywhere in the binding (no GPU)."""
import numpy as np
import pytest
import torch

import skinny_gemm_qlin_amd as ql

X = torch.zeros((2, 64), dtype=torch.bfloat16)
W = torch.zeros((8, 32), dtype=torch.uint8)
S = torch.zeros((8, 2), dtype=torch.bfloat16)
CALLS = {"gemv": (ql.qlin_gemv_w4, "x"), "gemv_bwd": (ql.qlin_gemv_w4_bwd, "dy"), "glu": (ql.qlin_glu_w4, "x"),
         "glu_bwd": (lambda *a: ql.qlin_glu_w4_bwd(*a, x=X), "dy")}


@pytest.mark.parametrize("bad", [None, 3, "x", [1.0], np.zeros((2, 64), np.float32)])
@pytest.mark.parametrize("call", CALLS)
def test_operands_that_are_no_tensors(call, bad):
    fn, first = CALLS[call]
    with pytest.raises(TypeError, match=f"{first}: expected a torch.Tensor"):
        fn(bad, W, S)
    for args in ((X, bad, S), (X, W, bad)):
        # of host tensors the first operand is refused for its device before the others are looked at
        with pytest.raises((TypeError, ValueError), match="expected a torch.Tensor|device"):
            fn(*args)


@pytest.mark.parametrize("bad", [3, "y", [1.0]])
def test_outputs_that_are_no_tensors(bad):
    with pytest.raises(TypeError, match="y: expected a torch.Tensor"):
        ql._out16(bad, "y", X, 2, 8)
    with pytest.raises(TypeError, match="workspace: expected a torch.Tensor"):
        ql._w4_workspace(bad, 1, 65536, 1024, X, None)
