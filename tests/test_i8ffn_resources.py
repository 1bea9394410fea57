"""What the compiler made of the INT8 feed-forward kernels, from the metadata of the built library (no GPU)."""
from test_w4_resources import kernels  # noqa: F401


def test_few_token_kernels(kernels):  # noqa: F811
    """Nothing in private memory (its loads queue behind the weights' and are waited for with them), and registers for
    the eight waves of a workgroup, two on each SIMD."""
    few = [k for n, k in kernels.items() if "few_front_kernel" in n or "few_down_kernel" in n]
    assert few
    assert not any(k[".private_segment_fixed_size"] for k in few) and max(k[".vgpr_count"] for k in few) <= 256


def test_matrix_kernels(kernels):  # noqa: F811
    gemm = [k for n, k in kernels.items() if "i8_gemm_kernel" in n]
    assert gemm and not any(k[".private_segment_fixed_size"] or k[".vgpr_spill_count"] for k in gemm)
