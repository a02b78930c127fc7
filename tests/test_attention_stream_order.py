"""The attention operators' kernels start while the kernel ahead of them may still write: they wait for it, and read by ordinary loads
and copies what it may write. A check of the sources; runs without a GPU."""
import os
import re

import pytest

from weight_only_quantized_wq4_gb300 import builder


def code(name):
    with open(os.path.join(builder.CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("name", ["wq4_append.cu", "wq4_tree_attention.cu", "wq4_attention_tiles.cu", "wq4_verify.cu"])
def test_kernels_wait_and_use_ordinary_loads(name):
    text = code(name)
    for kernel in text.split("__global__")[1:]:
        assert "griddepcontrol.wait" in kernel and "__restrict" not in kernel
    assert not re.findall(r"__ldg|\.global(?:\.\w+)*\.nc", text + code("wq4_attention.cuh") + code("wq4_cache.cuh"))
