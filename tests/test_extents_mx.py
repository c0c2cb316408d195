"""Sizes and extents of the block-scaled kernels, checked on the CPU through the functions that the
kernels and their launchers call (csrc/tile_addressing.h; `extent_check_mx.cpp`)."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "tests", "extent_check_mx.cpp")
CSRC = os.path.join(ROOT, "register_tiled_matrix_amd", "csrc")


@pytest.fixture(scope="module")
def checker(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    out = str(tmp_path_factory.mktemp("extent_mx") / "extent_check_mx")
    subprocess.run([gxx, "-O2", "-std=c++17", "-Wall", "-Werror", "-Wno-unused-function", f"-I{CSRC}", SRC, "-o", out],
                   check=True, capture_output=True, text=True)
    return out


def _run(exe, *args):
    r = subprocess.run([exe, *map(str, args)], capture_output=True, text=True, timeout=300)
    return r.returncode, r.stdout


@pytest.mark.parametrize("cols", [1, 7, 8, 9, 777, 2**31 - 9, 2**31 - 8, 2**31 - 7, 2**31 - 1])
def test_units_of_a_converted_row(checker, cols):
    rc, out = _run(checker, "units", cols)
    assert rc == 0 and out == f"{-(-cols // 8)} units\n", out


def test_kernel_and_launch_count_units_alike():
    # nothing in the conversions rounds columns up to units by itself
    text = open(os.path.join(CSRC, "mx_convert.hip")).read()
    assert "+ 7) / 8" not in text and text.count("addr::mx_units(") == 3


@pytest.mark.parametrize("fp4", [0, 1])
@pytest.mark.parametrize("cols", [1, 2, 33, 2**31 - 2, 2**31 - 1])
def test_bytes_of_a_row_of_codes(checker, fp4, cols):
    rc, out = _run(checker, "bytes", fp4, cols)
    assert rc == 0 and out == f"{-(-cols // 2) if fp4 else cols} bytes\n", out


@pytest.mark.parametrize("source", sorted(n for n in os.listdir(CSRC) if "mx_" in n and n.endswith(".hip")))
def test_no_kernel_rounds_a_row_up_in_32_bits(source):
    # cols + 1 passes 2^31 at the widest rows; the sizes come from the functions above
    assert "cols + 1) / 2" not in open(os.path.join(CSRC, source)).read()


# (order, M, N, K, lda, ldc); 256-wide tiles in parts where 33 to 128 of them meet K >= 8192
WIDE = [
    ("nt", 300, 8448, 8288, 8288, 8448),
    ("nt", 300, 8448, 8288, 2**22 - 8, 8448),        # the longest rows that leave 256 of them below 2^31 bytes
    ("nt", 300, 8448, 8288, 5 * 2**20, 8448),        # 128-wide tiles from there on
    ("nn", 300, 8448, 8296, 2**23 - 8, 8448),
    ("tn", 1040, 1824, 8288, 1040, 1824),
    ("tt", 1040, 1824, 8288, 1048, 1830),
]


@pytest.mark.parametrize("case", WIDE, ids=lambda c: "-".join(map(str, c)))
def test_descriptor_accesses_stay_inside_the_operands(checker, case):
    rc, out = _run(checker, "one", *case)
    assert rc == 0 and out.startswith("taken 1 "), out


@pytest.mark.parametrize("case", WIDE[2:4], ids=lambda c: "-".join(map(str, c)))
def test_wide_tiles_do_not_reach_that_far(checker, case):
    # why these stay on 128-wide tiles: the offsets that stand for "past K" wrap on 256-wide ones
    rc, out = _run(checker, "force", *case)
    assert rc == 1 and "wraps past 2^32" in out, out


def test_seeded_sweep(checker):
    rc, out = _run(checker, "sweep", 20261206, 120)
    assert rc == 0 and int(out.split()[1]) > 20, out
