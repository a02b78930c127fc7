"""Where the compiler gives the attention kernel for many rows other registers than its warps count on: which counts it can run with,
and that a call goes to the other kernel if it cannot. Runs without a GPU."""
import os
import shutil
import subprocess

import pytest

from weight_only_quantized_wq4_gb300 import builder

DRIVER = r"""
#include <cstdio>
#include <cstdlib>
#include "wq4_check.h"
int main(int, char** v) {
    std::printf("%d\n", wq4::check::registers_cover(std::atoi(v[1]), 640, 128 * 64 + 512 * 104) ? 1 : 0);
    return 0;
}
"""


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no g++")
    at = tmp_path_factory.mktemp("registers")
    src, out = str(at / "registers.cpp"), str(at / "registers")
    with open(src, "w") as f:
        f.write(DRIVER)
    r = subprocess.run([gxx, "-std=c++17", "-I", builder.CSRC, src, "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return out


@pytest.mark.parametrize("regs,fits", [(96, 1), (95, 1), (89, 1), (88, 0), (80, 0), (97, 1), (102, 1)])
def test_registers_are_given_out_in_eights(exe, regs, fits):
    assert subprocess.run([exe, str(regs)], capture_output=True, text=True).stdout.strip() == str(fits)


def test_the_call_asks_before_it_chooses():
    with open(os.path.join(builder.CSRC, "wq4_tree_attention.cu")) as f:
        call = f.read().split("int wq4_tree_attention(")[1]
    assert call.index("attention_tiles_fit(") < call.index("a.box =") < call.index("launch_attention_tiles(")
    with open(os.path.join(builder.CSRC, "wq4_attention_tiles.cu")) as f:
        assert "WQ4_ERR_CUDA" not in f.read()
