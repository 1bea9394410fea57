"""The block cases of the INT8 expert layer's down projection reach what they are meant to reach (no GPU)."""
import os
import subprocess

import pytest

from conftest import ROOT
from i8ffn_block_cases import CASES

NAMES = ("fits", "own_codes", "pairs", "most", "block", "rows", "chunk")


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("i8ffn") / "blocks")
    subprocess.run(["g++", "-O2", "-std=c++17", os.path.join(ROOT, "tests", "i8ffn_blocks.cpp"), "-o", out], check=True)

    def run(M, H, I, topk, E):
        text = subprocess.run([out, *map(str, (M, H, I, topk, E))], capture_output=True, text=True, check=True).stdout
        return dict(zip(NAMES, map(int, text.split())))
    return run


@pytest.mark.parametrize("M,E,topk,H,I,whole", CASES)
def test_cases_have_several_blocks(plan, M, E, topk, H, I, whole):
    p = plan(M, H, I, topk, E)
    assert p["fits"] and p["block"] < p["most"]
    assert (p["pairs"] <= p["rows"]) == whole


def test_both_sources_of_codes_are_there(plan):
    assert {plan(M, H, I, topk, E)["own_codes"] for M, E, topk, H, I, _ in CASES} == {0, 1}


@pytest.mark.parametrize("H", [16, 1024, 1040, 4112, 7168, 131072])
def test_sums_have_room(plan, H):
    """Every block's sums are inside their part of LDS, and no workgroup is without a row group."""
    for M, topk in ((1, 1), (3, 5), (16, 15), (16, 16)):
        p = plan(M, H, 16, topk, 8)
        assert 1 <= p["block"] <= p["most"] and p["block"] * p["pairs"] * 16 <= 16 * 1024
        assert p["most"] == -(-(H // 4) // min(H // 4, 256))
