"""How the 4-bit weight calls are laid out, from the host code that decides it (no GPU)."""
import os
import subprocess

import pytest

from conftest import ROOT


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    """plan([(M, K, group, C, gated), ...]) -> [[kernel, numbers ...], ...]"""
    exe = str(tmp_path_factory.mktemp("plan") / "w4_plan")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", os.path.join(ROOT, "skinny_gemm_qlin_amd", "csrc"),
                    os.path.join(ROOT, "tests", "w4_plan.cpp"), "-o", exe], check=True)

    def run(calls):
        text = "".join(f"{m} {k} {g} {c} {int(gated)}\n" for m, k, g, c, gated in calls)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout
        return [[f if i == 0 else int(f) for i, f in enumerate(line.split())] for line in out.splitlines()]
    return run


def test_kernels_by_size(plan):
    """Up to 16 tokens the decode kernels, up to 64 and on small matrices the mid kernel, then the GEMM."""
    got = [p[0] for p in plan([(1, 5120, 128, 17408, False), (16, 4096, 128, 14336, True), (17, 5120, 128, 17408, False),
                               (64, 5120, 128, 17408, False), (128, 7168, 128, 4096, False), (2048, 5120, 128, 17408, False),
                               (2048, 4096, 128, 14336, True)])]
    assert got == ["few", "few", "mid", "mid", "mid", "gemm", "gemm"]


def _mid_lds(tokens, ntl, stages, groups):
    """LDS of the mid kernel: stages of 256 K of its token and code rows, the scales of 32 ntl rows."""
    rows = 32 if tokens <= 32 else 48 if tokens <= 48 else 64
    return stages * (rows * 512 + ntl * 32 * 128) + 256 + 3 * 32 * ntl * groups + 128


@pytest.mark.parametrize("M", [17, 32, 33, 48, 49, 64])
def test_many_scales_keep_the_mid_kernel(plan, M):
    """17 to 64 tokens: as many stages as fit next to the scales, down to two, before the GEMM takes the call."""
    groups = list(range(400, 1400, 4))
    got = plan([(M, 32 * g, 32, 8192, False) for g in groups])
    seen = set()
    for g, p in zip(groups, got):
        if _mid_lds(M, 1, 2, g) <= 160 * 1024:
            assert p[0] == "mid", (g, p)
            seen.add(p[2])
            assert _mid_lds(M, p[1], p[2], g) <= 160 * 1024
            if p[2] == 2:  # only where three do not fit
                assert p[1] == 1 and _mid_lds(M, 1, 3, g) > 160 * 1024
        elif p[0] == "mid":
            raise AssertionError((g, p))
    assert 2 in seen and 3 in seen
    assert plan([(64, 28672, 32, 8192, False)])[0][:3] == ["mid", 1, 2]  # a down projection in groups of 32


@pytest.mark.parametrize("gated", [False, True])
def test_rows_that_decode_without_rounding(plan, gated):
    """The decode kernels take rows of as many groups as the header promises unrounded weights for."""
    calls, want = [], []
    for M in range(1, 17):
        most = (2600 if M <= 8 else 1290) if gated else (5300 if M <= 8 else 2600)
        for group in (32, 64, 96, 128, 192, 384):
            for groups in (most, most - 1, most - 77, most // 2):
                if group * groups <= 1 << 20:
                    calls += [(M, group * groups, group, C, gated) for C in (1, 500, 20000)]
    assert all(p[0] == "few" for p in plan(calls))
    # far past it they cannot: the scales of one tile fill LDS
    assert all(p[0] != "few" for p in plan([(M, 32 * 7000, 32, 500, gated) for M in range(1, 17)]))


def test_layouts_fit(plan):
    """What a decode call is given fits LDS, its waves a workgroup and its passes the row."""
    calls = [(M, group * groups, group, C, gated) for M in (1, 2, 5, 8, 9, 12, 16) for group in (32, 128, 160)
             for groups in (1, 3, 40, 41, 300, 1200) for C in (1, 9, 4099, 17408, 300000) for gated in (False, True)]
    for (M, K, group, C, gated), p in zip(calls, plan(calls)):
        assert p[0] == "few"
        _, pl, nw, passes, rows, depth, lds = p
        assert 1 <= nw <= 16 and pl in (1, 2) and depth in (1, 2) and lds <= 160 * 1024 and rows >= 8
        assert nw * pl * passes * 256 >= K > nw * pl * (passes - 1) * 256
