"""The 4-bit custom operators around their kernels (no GPU)."""
import torch

from skinny_gemm_qlin_amd import torch_ops


def _seen(monkeypatch, op, dy):
    """The gradient that the binding's call gets from the operator."""
    got = []
    name = "qlin_glu_w4_bwd" if op is torch_ops.glu_w4_bwd else "qlin_gemv_w4_bwd"

    def call(t, w, s, z, **k):
        got.append(t)
        rows, width = t.shape[0], 2 * w.shape[1]
        dx = t.new_zeros((rows, width))
        return (dx, t.new_zeros((rows, w.shape[0]))) if op is torch_ops.glu_w4_bwd else dx

    monkeypatch.setattr(torch_ops, name, call)
    rows = dy.shape[1] * (2 if op is torch_ops.glu_w4_bwd else 1)
    w, s = torch.zeros((rows, 32), dtype=torch.uint8), torch.zeros((rows, 2), dtype=dy.dtype)
    x = torch.zeros((dy.shape[0], 64), dtype=dy.dtype)
    op(dy, w, s, None, x) if op is torch_ops.glu_w4_bwd else op(dy, w, s)
    return got[0]


def test_gradients_that_the_kernels_read_as_they_are(monkeypatch):
    """The gates take any row pitch; only a matrix product needs aligned rows."""
    odd = torch.randn(5, 33, dtype=torch.float16)
    even = torch.randn(5, 40, dtype=torch.float16)
    assert _seen(monkeypatch, torch_ops.glu_w4_bwd, odd).data_ptr() == odd.data_ptr()
    assert _seen(monkeypatch, torch_ops.glu_w4_bwd, even[1:, 1:]).data_ptr() == even[1:, 1:].data_ptr()
    assert _seen(monkeypatch, torch_ops.gemv_w4_bwd, even).data_ptr() == even.data_ptr()


def test_gradients_that_are_copied(monkeypatch):
    """Unaligned rows ahead of a matrix product; expanded and transposed ones everywhere."""
    odd = torch.randn(5, 33, dtype=torch.float16)
    for op in (torch_ops.gemv_w4_bwd, torch_ops.glu_w4_bwd):
        for dy in (odd[:1].expand(5, 33), odd[:, :1].expand(5, 16), odd.t()):
            got = _seen(monkeypatch, op, dy)
            assert torch.equal(got, dy) and got.stride(1) == 1 and got.stride(0) % 8 == 0 and got.data_ptr() % 16 == 0
    for dy in (odd, torch.randn(5, 48, dtype=torch.float16)[:, 1:41]):
        got = _seen(monkeypatch, torch_ops.gemv_w4_bwd, dy)
        assert torch.equal(got, dy) and got.stride(0) % 8 == 0 and got.data_ptr() % 16 == 0
