"""Rows past a tile's last, gathered rows and scales of the 8-bit float tiles: where their loads go, checked on the CPU through
the functions that the kernels call (csrc/tile_addressing.h; extent_check_f8_rows.cpp)."""
from __future__ import annotations

import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "tests", "extent_check_f8_rows.cpp")
CSRC = os.path.join(ROOT, "register_tiled_matrix_amd", "csrc")


@pytest.fixture(scope="module")
def checker(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    out = str(tmp_path_factory.mktemp("extent_f8_rows") / "extent_check_f8_rows")
    subprocess.run([gxx, "-O2", "-std=c++17", "-Wall", "-Werror", "-Wno-unused-function", f"-I{CSRC}", SRC, "-o", out], check=True,
                   capture_output=True, text=True)

    def run(*args):
        r = subprocess.run([out, *map(str, args)], capture_output=True, text=True, timeout=120)
        return r.returncode, r.stdout.strip()

    return run


@pytest.mark.parametrize("tile", [64, 128, 256])
@pytest.mark.parametrize("mode,rows,K,ld", [
    ("rows", 256, 1, 16), ("rows", 256, 777, 784), ("rows", 256, 8191, 8192), ("rows", 256, 8355000, 8355008),  # 256 ld + K + 128 just below 2^31
    ("rows", 3, 129, 144),
    ("gather", 1, 1, 16), ("gather", 1, 2**30 - 144, 2**30), ("gather", 37, 777, 784), ("gather", 4096, 2048, 2048), ("gather", 4096, 2000, 2064),
    ("gather", 100000, 21000, 21008), ("gather", 2**27 - 20, 1, 16)])  # all rows just below 2^31
def test_rows_past_the_last_are_not_loaded(checker, mode, rows, K, ld, tile):
    assert checker(mode, rows, K, ld, tile) == (0, "ok")


@pytest.mark.parametrize("rows,K,ld", [(2**27, 1, 16), (300000, 8000, 8000), (1, 2**30, 2**30), (1, 2**31 - 129, 2**31 - 128)])
def test_gathered_rows_out_of_reach_are_not_taken(checker, rows, K, ld):
    assert checker("gather", rows, K, ld, 128) == (0, "not taken")


@pytest.mark.parametrize("rows,blocks,s_row,s_col", [
    (1, 1, 1, 1), (8192, 64, 1, 8192), (8192, 64, 64, 1), (64, 64, 64, 1), (300, 5, 0, 0), (1, 64, 2**20, 0), (2**22 - 1, 127, 1, 2**22),
    (2**22 - 1, 127, 128, 1), (1, 2**22, 1, 127), (5, 2, 2**26, 2**26)])
def test_scales_are_where_their_strides_say(checker, rows, blocks, s_row, s_col):
    assert checker("scales", rows, blocks, s_row, s_col) == (0, "ok")


@pytest.mark.parametrize("rows,blocks,s_row,s_col", [(2**22, 127, 1, 2**22), (2**22, 128, 1, 2**22), (2**22, 128, 128, 1), (4, 4, 2**27, 1), (1, 1, 1, 2**29)])
def test_scales_out_of_reach_are_not_taken(checker, rows, blocks, s_row, s_col):
    assert checker("scales", rows, blocks, s_row, s_col) == (0, "not taken")


def test_seeded_sizes(checker):
    rng = random.Random(20261209)
    for _ in range(60):
        rows, K = rng.randint(1, 900), rng.randint(1, 900)
        ld = -(-K // 16) * 16 + 16 * rng.randint(0, 3)
        assert checker(rng.choice(["rows", "gather"]), rows, K, ld, rng.choice([64, 128, 256])) == (0, "ok"), (rows, K, ld)
        blocks, pad = rng.randint(1, 300), rng.randint(0, 9)
        by_rows = rng.random() < 0.5
        assert checker("scales", rows, blocks, blocks + pad if by_rows else 1, 1 if by_rows else rows + pad) == (0, "ok"), (rows, blocks, pad)
