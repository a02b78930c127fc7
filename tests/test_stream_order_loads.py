"""Kernels that start while the kernel ahead of them still runs (programmatic dependent launch) read what that kernel may write by
ordinary loads: read-only ones (`__ldg`, `ld.global.nc`, `const __restrict__` parameters) ask for data that nothing writes while
the kernel is there. A check of the sources; runs without a GPU."""
import os
import re

import pytest

from weight_only_quantized_wq4_gb300 import builder


def code(name):
    with open(os.path.join(builder.CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("name", ["wq4_rows.cu", "wq4_block_mm.cu", "wq4_logprobs.cu", "wq4_api.cu"])
def test_no_read_only_loads(name):
    text = code(name)
    assert "griddepcontrol.wait" in text
    assert not re.findall(r"__ldg|\.global(?:\.\w+)*\.nc", text)
    for kernel in text.split("__global__")[1:]:
        assert "griddepcontrol" not in kernel or "__restrict" not in kernel
