"""Which form the dense layer takes (csrc/linear_bounds.hpp, built here with g++): large tiles only where rows fill them."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# rows, columns, whether the large tiles were the faster form when both were measured (within 7 %: None)
MEASURED = [(17, 32768, False), (32, 32768, False), (64, 32768, False), (128, 32768, True), (192, 32768, True),
            (512, 32768, True), (17, 65536, False), (32, 65536, False), (64, 65536, True), (128, 65536, True),
            (17, 131072, False), (32, 131072, False), (64, 131072, None), (128, 131072, True), (384, 131072, True),
            (384, 16384, None), (512, 16384, True), (1100, 16384, True), (264, 24576, True), (1024, 8192, True),
            (2048, 4096, True), (4096, 2048, True), (8192, 4096, True), (8192, 16384, True), (1 << 20, 64, None)]


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    folder = tmp_path_factory.mktemp("forms")
    source, exe = str(folder / "rule.cpp"), str(folder / "rule")
    with open(source, "w") as f:
        f.write('#include "%s"\n#include <stdio.h>\n#include <stdlib.h>\n'
                "int main(int n, char **v) { for (int i = 1; i + 1 < n; i += 2) "
                'printf("%%d", mxfp4::tiles_filled(atoll(v[i]), atoll(v[i + 1]))); }\n'
                % os.path.join(ROOT, "block_scaled_mxfp4_bf16_amd", "csrc", "linear_bounds.hpp"))
    subprocess.check_call(["g++", "-std=c++17", "-Wall", "-o", exe, source])

    def of(sizes):
        return [c == "1" for c in subprocess.check_output([exe] + [str(v) for s in sizes for v in s], text=True)]
    return of


def test_the_faster_form_of_the_measured_sizes(rule):
    got = rule([(m, n) for m, n, _ in MEASURED])
    assert [(m, n, g) for (m, n, want), g in zip(MEASURED, got) if want is not None and g != want] == []


def test_many_rows_always_fill_them(rule):
    """From 512 rows on nothing but the number of tiles counts."""
    sizes = [(m, n) for m in (512, 513, 767, 1024, 1025, 8192, 100000) for n in (48, 4096, 16384, 16400, 65536, 1 << 20)
             if -(-m // 256) * -(-n // 256) >= 128]
    assert all(rule(sizes))


def test_the_kernels_are_chosen_by_it():
    with open(os.path.join(ROOT, "block_scaled_mxfp4_bf16_amd", "csrc", "linear_kernels.hip")) as f:
        assert "tiles_filled(a.M, a.N)" in f.read().split("static bool use_tiles")[1].split("}")[0]
