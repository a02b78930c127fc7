"""What wq4_get_last_error says of each bit that kernels record, compiled for the host. Runs without a GPU."""
import os
import re
import shutil
import subprocess

import pytest

import weight_only_quantized_wq4_gb300 as wq4
from weight_only_quantized_wq4_gb300 import builder

DRIVER = r"""
#include <cstdio>
#include <cstdlib>
#define __host__
#define __device__
#include "wq4_params.h"
int main(int, char** v) {
    std::printf("%d\n", wq4::status_error(static_cast<uint32_t>(std::atoi(v[1]))));
    return 0;
}
"""


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    gxx, nvcc = shutil.which("g++"), shutil.which("nvcc")
    if not gxx or not nvcc:
        pytest.skip("no g++ or no CUDA headers")
    at = tmp_path_factory.mktemp("status")
    src, out = str(at / "status.cpp"), str(at / "status")
    with open(src, "w") as f:
        f.write(DRIVER)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    r = subprocess.run([gxx, "-std=c++17", "-I", builder.CSRC, "-I", builder.INCLUDE, "-I", cuda, src, "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return out


@pytest.mark.parametrize("status,code", [(0, wq4.OK), (1, wq4.ERR_TIMEOUT), (2, wq4.ERR_INVALID), (4, wq4.ERR_BOUNDS), (8, wq4.ERR_INVALID),
                                         (16, wq4.ERR_CUDA), (17, wq4.ERR_TIMEOUT), (9, wq4.ERR_INVALID), (31, wq4.ERR_BOUNDS)])
def test_each_bit(exe, status, code):
    assert subprocess.run([exe, str(status)], capture_output=True, text=True).stdout.strip() == str(code)


def test_a_base_off_its_boundary_is_no_timeout():
    with open(os.path.join(builder.CSRC, "wq4_attention_tiles.cu")) as f:
        check = re.search(r"if \(s_base & 1023u\) \{(.*?)\n    \}", f.read(), flags=re.S).group(1)
    assert "kStatusPlacement" in check and "kStatusTimeout" not in check
