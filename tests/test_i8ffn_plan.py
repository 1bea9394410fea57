"""By which sizes the INT8 feed-forward calls choose their kernels, and the quotient of their quantiser (no GPU)."""
import os
import subprocess

import pytest

from conftest import ROOT

NAMES = ("fits", "quantise", "turn", "sets", "down_rows", "chunk", "tile_rows", "dense_tile", "large")


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("i8ffn") / "host")
    subprocess.run(["g++", "-O2", "-std=c++17", "-ffp-contract=off", "-mfma", os.path.join(ROOT, "tests", "i8ffn_host.cpp"),
                    "-o", out], check=True)
    return out


@pytest.fixture(scope="module")
def plan(exe):
    def run(M, K, I, topk=0, E=0):
        out = subprocess.run([exe, "plan", *map(str, (M, K, I, topk, E))], capture_output=True, text=True, check=True).stdout
        return dict(zip(NAMES, map(int, out.split())))
    return run


def test_quotients(exe):
    """Every mantissa of bf16 and fp16 against every scale that a largest magnitude can give: codes as by division."""
    assert subprocess.run([exe, "quotients"], capture_output=True, text=True, check=True).stdout.strip() == "0"


def test_kernels_by_size(plan):
    assert plan(1, 4096, 14336)["fits"] and plan(16, 5120, 8704)["fits"] and plan(1, 131072, 16)["fits"]
    assert not plan(17, 16, 16)["fits"] and not plan(16, 14336, 16)["fits"] and not plan(2, 131072, 16)["fits"]
    assert [plan(M, 7168, 2048, 6, 64)["sets"] for M in (1, 4, 5, 8, 13, 16)] == [1, 1, 1, 2, 2, 4]
    assert [plan(M, 4096, 14336)["sets"] for M in (1, 4, 5, 8, 9, 16)] == [1, 1, 2, 2, 4, 4]
    assert [plan(1, K, 16)["turn"] for K in (16, 768, 1024, 1536, 2048, 2064, 4096, 5120, 7168, 14336)] == [
        3, 3, 4, 3, 4, 3, 4, 4, 4, 4]
    assert [plan(M, 7168, 2048, 6, 64)["tile_rows"] for M in (64, 171, 597, 598)] == [32, 64, 64, 128]
    small, wide, square, two = range(4)  # 64 x 64, 64 x 128, 128 x 128 with a ring of four, of two
    assert [plan(M, 4096, 14336)["dense_tile"] for M in (17, 64, 65, 128, 129, 256, 257)] == [
        wide, wide, square, square, two, two, square]
    assert [plan(M, 7168, 4096)["dense_tile"] for M in (17, 64, 128, 129, 256, 257)] == [
        small, small, small, wide, wide, square]
    assert plan(1023, 4096, 14336)["large"] == 0 and plan(2048, 4096, 14336)["large"] == 96 * 128


@pytest.mark.parametrize("I", [16, 768, 2048, 14336, 32768, 131072 - 16, 131072])
def test_the_down_projection_always_has_room(plan, I):
    """At least one row of codes, chunks no larger than the rows, and both parts of LDS inside it."""
    for M, topk, E in ((1, 1, 1), (2, 2, 2), (16, 16, 16), (16, 8, 128), (13, 5, 1024), (16, 16, 1)):
        p = plan(M, 16, I, topk, E)
        assert 1 <= p["chunk"] <= min(16, p["down_rows"]) and p["down_rows"] <= M * topk
        turn = 256 * plan(1, I, 16)["turn"]
        pitch = (I + turn - 1) // turn * turn + 64
        assert p["down_rows"] * pitch <= 130 * 1024


def test_whole_rounds_of_large_tiles(plan):
    for M in (1024, 1500, 2048, 4096, 16384):
        for I in (128, 1000, 2051, 14336):
            large, mt = plan(M, 4096, I)["large"], (M + 255) // 256
            assert large % 128 == 0 and 0 <= large <= I
            assert -(mt * (large // 128)) % 256 < mt  # workgroups that the last round lacks: less than a column of tiles
