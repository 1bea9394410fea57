"""The gated gradient in place, as far as the host can tell (no GPU): pointers are never dereferenced."""
import os

import pytest

A = 0x10000


@pytest.fixture(scope="module")
def q():
    from skinny_gemm_qlin_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from skinny_gemm_qlin_amd import _build
        _build.build()
    return _lib.load()


def test_gate_gradient_over_gu_at_another_pitch(q):
    """dgu may be gu itself; at another row pitch a row would be written before it is read.  One row has no pitch."""
    def call(M, ldgu, lddgu):
        return q.qlin_glu_w4_bwd(A, 32, M, 32, 0, 0, None, 0, A, ldgu, A, 512, 1024, A, None, 128, A, lddgu, A, 1024,
                                 None, 0, None)
    assert call(2, 64, 72) == -3 and call(2, 72, 64) == -3 and call(2, 128, 64) == -3
    # past that check: the workspace that these sizes need is missing
    big = 32768
    def wide(M, ldgu, lddgu):
        return q.qlin_glu_w4_bwd(A, big, M, big, 0, 0, None, 0, A, ldgu, A, 512, 1024, A, None, 128, A, lddgu, A, 1024,
                                 None, 0, None)
    assert wide(2, 2 * big, 2 * big) == -5 and wide(1, 2 * big, 2 * big + 8) == -5 and wide(2, 2 * big, 2 * big + 8) == -3
