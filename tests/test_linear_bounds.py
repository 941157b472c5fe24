"""The offsets that the dense layer's kernels read a prepared matrix at stay
below 2^31 up to the largest one (csrc/linear_bounds.hpp, built here with g++,
once with the undefined-behaviour checks)."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_scaled_mxfp4_bf16_amd", "csrc")


@pytest.mark.parametrize("extra", [["-O1"], ["-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all"]])
def test_offsets_stay_below_2_31(tmp_path, extra):
    exe = str(tmp_path / "check")
    subprocess.check_call(["g++", "-std=c++17", "-Wall", *extra, "-o", exe, os.path.join(ROOT, "tests", "linear_bounds_check.cpp")])
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "bounds ok" in r.stdout


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def test_the_kernels_read_the_weights_through_them():
    tile, split = source("linear_tile.hip"), source("linear_kernels.hip")
    assert "u.b_off[q] = group_within(g, N >> 4) * K * 8;" in tile and "steps = tile_steps(K)" in tile
    assert re.search(r"gw\[nt\] = group_within\(gw\[nt\], groups\)", split)
    assert re.search(r"static bool use_tiles[^}]*tile_offsets_fit\(a\.N, a\.K\)", split)
