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
