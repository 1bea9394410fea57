"""The differentiable 4-bit operators under torch's tracing of forward and backward."""
import pytest
import torch

from gpu_util import lib, need_gpu
from w4_util import dev_w, gen_w4, gen_x

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def layer():
    need_gpu()
    lib()
    import skinny_gemm_qlin_amd.torch_ops  # noqa: F401
    return dev_w(*gen_w4(64, 128, 32, "bf16", True, seed=1))


def test_operator_checks(layer):
    """Schema, autograd registration, fake tensors, tracing with dynamic shapes: with and without a gradient."""
    for grad in (False, True):
        x = gen_x(20, 128, "bf16", 1).cuda().requires_grad_(grad)
        torch.library.opcheck(torch.ops.qlin.gemv_w4.default, (x, *layer))
        torch.library.opcheck(torch.ops.qlin.glu_w4.default, (x, *layer, 1, False))
    x = x.detach()
    torch.library.opcheck(torch.ops.qlin.glu_w4.default, (x, *layer, 1, True))
    torch.library.opcheck(torch.ops.qlin.gemv_w4_bwd.default, (gen_x(20, 64, "bf16", 2).cuda(), *layer))
    torch.library.opcheck(torch.ops.qlin.glu_w4_bwd.default, (gen_x(20, 32, "bf16", 2).cuda(), *layer, x, None, 1))


@pytest.mark.parametrize("M", [3, 40, 130])
def test_compiled_gradients(layer, M):
    """A compiled function that returns both outputs, and one that keeps gate and up for itself."""
    def both(x):
        return torch.ops.qlin.glu_w4(x, *layer, 1, False)

    def kept(x):
        return (torch.ops.qlin.glu_w4(x, *layer, 0, True)[0],)

    x = gen_x(M, 128, "bf16", 1).cuda().requires_grad_(True)
    dy = gen_x(M, 32, "bf16", 2).cuda()
    for fn in (both, kept):
        (want,) = torch.autograd.grad(fn(x)[0], x, dy)
        y = torch.compile(fn, backend="aot_eager", fullgraph=True)(x)[0]
        (got,) = torch.autograd.grad(y, x, dy)
        assert torch.equal(got, want)
