"""What the second launch of an expert operator reads from the workspace stays
within its own call's sizes whatever is there (csrc/experts_bounds.hpp, built
here with g++, once with the undefined-behaviour checks)."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_scaled_mxfp4_bf16_amd", "csrc")


@pytest.mark.parametrize("extra", [["-O1"], ["-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all"]])
def test_units_stay_within_the_call(tmp_path, extra):
    exe = str(tmp_path / "check")
    subprocess.check_call(["g++", "-std=c++17", "-Wall", *extra, "-o", exe, os.path.join(ROOT, "tests", "experts_bounds_check.cpp")])
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "bounds ok" in r.stdout


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def test_the_kernels_read_the_workspace_through_it():
    device, tile, route = source("grouped_device.hpp"), source("grouped_tile.hpp"), source("route_kernels.hip")
    assert re.search(r"return unit_of\(", device) and re.search(r"return within\(.*, 0, a\.max_units\)", device)
    assert "tile_place(" in tile
    # the router's places and its number of used places
    assert re.search(r"if \(\(unsigned\)at < \(unsigned\)pairs\)", route)
    assert len(re.findall(r"used = within\(n, 0, ", route)) == 2
