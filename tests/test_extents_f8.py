"""Where the 8-bit float tiles read, checked on the CPU through the functions that the kernels and their launches call
(csrc/tile_addressing.h; extent_check_f8.cpp)."""
from __future__ import annotations

import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "tests", "extent_check_f8.cpp")
CSRC = os.path.join(ROOT, "register_tiled_matrix_amd", "csrc")


@pytest.fixture(scope="module")
def checker(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    out = str(tmp_path_factory.mktemp("extent_f8") / "extent_check_f8")
    subprocess.run([gxx, "-O2", "-std=c++17", "-Wall", "-Werror", "-Wno-unused-function", f"-I{CSRC}", SRC, "-o", out], check=True,
                   capture_output=True, text=True)

    def run(order, rows, cols, ld, tile):
        r = subprocess.run([out, order, *map(str, (rows, cols, ld, tile))], capture_output=True, text=True, timeout=120)
        return r.returncode, r.stdout.strip()

    return run


@pytest.mark.parametrize("tile", [64, 128, 256])
@pytest.mark.parametrize("order,rows,cols,ld", [
    ("kc", 1, 1, 16), ("kc", 1, 128, 128), ("kc", 300, 777, 784), ("kc", 257, 129, 144), ("kc", 64, 8191, 8192), ("kc", 513, 1504, 4096),
    ("kc", 700, 8355000, 8355008),                  # 256 ld + K + 128 just below 2^31
    ("nn", 1, 1, 16), ("nn", 128, 16, 16), ("nn", 777, 300, 304), ("nn", 129, 257, 272), ("nn", 8191, 513, 528),
    ("nn", 4000, 100, 520208)])
def test_loads_stay_in_chunks_of_the_matrix_and_fill_their_slots(checker, order, rows, cols, ld, tile):
    assert checker(order, rows, cols, ld, tile) == (0, "ok")


@pytest.mark.parametrize("order,rows,cols,ld", [("kc", 700, 2**23, 2**23), ("nn", 2**16, 2**15 - 16, 2**15)])
def test_operands_out_of_reach_are_not_taken(checker, order, rows, cols, ld):
    assert checker(order, rows, cols, ld, 256) == (0, "not taken")


def test_seeded_sizes(checker):
    rng = random.Random(20261208)
    for _ in range(60):
        rows, cols = rng.randint(1, 900), rng.randint(1, 900)
        ld = -(-cols // 16) * 16 + 16 * rng.randint(0, 3)
        order, tile = rng.choice(["kc", "nn"]), rng.choice([64, 128, 256])
        assert checker(order, rows, cols, ld, tile) == (0, "ok"), (order, rows, cols, ld, tile)
