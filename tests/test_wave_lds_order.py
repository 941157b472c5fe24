"""The 128-row product's tiles turn their sums in LDS: lanes of a wave write
16 bytes that other lanes of it read, and the next rows write over them.  In
program order a fence has to stand between the write and the read and between
the read and the next write, since the compiler may otherwise move one past the
other: a lane's own addresses differ.  Checked in the code as it goes into the
optimizer (device pass of hipcc, no GPU)."""
import os
import re
import subprocess

import pytest

from block_scaled_mxfp4_bf16_amd import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def functions(tmp_path_factory):
    hipcc = build.hipcc()
    if not os.path.exists(hipcc):
        pytest.skip("no hipcc")
    out = str(tmp_path_factory.mktemp("ir") / "grouped.ll")
    subprocess.check_call([hipcc, *build.HIPCC_FLAGS, "--cuda-device-only", "-S", "-emit-llvm", "-Xclang",
                           "-disable-llvm-passes", os.path.join(build.CSRC, "grouped_kernels.hip"), "-o", out],
                          stderr=subprocess.DEVNULL)
    with open(out) as f:
        text = f.read()
    return dict(re.findall(r"^define [^\n]*?@(\w+)\([^\n]*\{\n(.*?)^\}", text, re.M | re.S))


def test_turned_rows_are_fenced(functions):
    store = re.compile(r"_ZZN5mxfp419grouped_tile_kernelILb[01]E.*RKNS_4UnitE\w*$")
    names = [n for n in functions if store.match(n) and not n.startswith("_ZZZ")]
    assert len(names) == 4  # gated or not, wide stores or not
    for name in names:
        events = []
        for line in functions[name].splitlines():
            m = re.search(r"call .*@(\w+)\(", line)
            if m and m.group(1).startswith("_ZZZN5mxfp419grouped_tile_kernel"):
                events.append("address")
            elif m and "wave_lds_fence" in m.group(1):
                events.append("fence")
        assert events == ["address", "fence", "address", "fence"], (name, events)


def test_the_fence_is_one(functions):
    body = [b for n, b in functions.items() if "wave_lds_fence" in n]
    assert len(body) == 1
    assert 'fence syncscope("wavefront") acq_rel' in body[0] and "llvm.amdgcn.wave.barrier" in body[0]
