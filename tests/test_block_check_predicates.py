"""The block-scaled product's bounds predicate (csrc/wq4_check.h), compiled for the host and checked at its
boundaries: a copy starts inside the blocks of K and inside the rows of its tiles. Runs without a GPU."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "weight_only_quantized_wq4_gb300", "csrc")
OUT = os.path.join(ROOT, "weight_only_quantized_wq4_gb300", "_build", "check_host")

DRIVER = r"""
#include <cstdio>
#include <cstdlib>
#include "wq4_check.h"
int main(int, char** v) {
    std::printf("%d\n", wq4::check::block_copy_ok(std::atoll(v[1]), std::atoll(v[2]), std::atoll(v[3]), std::atoll(v[4])) ? 1 : 0);
    return 0;
}
"""


@pytest.fixture(scope="module")
def exe():
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no g++")
    os.makedirs(OUT, exist_ok=True)
    src, out = os.path.join(OUT, "block_check.cpp"), os.path.join(OUT, "block_check")
    with open(src, "w") as f:
        f.write(DRIVER)
    r = subprocess.run([gxx, "-std=c++17", "-I", CSRC, src, "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return out


@pytest.mark.parametrize("args,ok", [((0, 1, 0, 128), 1), ((16, 17, 3968, 4096), 1), ((17, 17, 0, 128), 0), ((-1, 17, 0, 128), 0),
                                     ((0, 1, 128, 128), 0), ((0, 1, -1, 128), 0), ((0, 0, 0, 128), 0)])
def test_block_copy(exe, args, ok):
    assert subprocess.run([exe, *map(str, args)], capture_output=True, text=True).stdout.strip() == str(ok)
