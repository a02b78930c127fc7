"""No attention kernel reads or writes global memory ahead of its wait for the kernel before it: a check of the sources, which sees a read
that is moved there. Runs without a GPU."""
import re

import pytest

from tests.test_attention_stream_order import code

FILES = ["wq4_append.cu", "wq4_tree_attention.cu", "wq4_attention_tiles.cu", "wq4_verify.cu"]
WAIT = 'asm volatile("griddepcontrol.wait;"'
# an argument's pointer indexed, added to, dereferenced or handed on; the schedule, which reads lengths; copies and loads
TOUCHES = re.compile(r"\ba\.\w+\s*\[|\ba\.(?:q|k|v|out|lse|table|starts|context|mask|cache|slots|positions|inv_freq|counters|stats|parts|"
                     r"q_out|q_weight|k_weight|logits|tokens|parents|draft_probs|temperature|uniforms|final_uniforms|accepted|path|"
                     r"next_tokens|status)\b|\bWalk\s+\w+\(|\.begin\(|\bbring\(|\btma_load|cp\.async|ld\.global|st\.global|__ldcg|__stcg|\batomic")


def ahead_of_the_wait(text):
    """The bodies of a source's kernels up to their wait."""
    out = []
    for kernel in text.split("__global__")[1:]:
        body = kernel[kernel.index("{"):]
        assert WAIT in body
        out.append(body[:body.index(WAIT)])
    return out


@pytest.mark.parametrize("name", FILES)
def test_nothing_is_read_ahead_of_the_wait(name):
    parts = ahead_of_the_wait(code(name))
    assert parts
    for part in parts:
        # (tensor maps are arguments, in constant memory)
        found = TOUCHES.findall(re.sub(r"prefetch_tensormap\(&a\.\w+\);", "", part))
        assert not found, found


@pytest.mark.parametrize("name,read", [
    ("wq4_append.cu", "const int heads = a.Hq + 2 * a.Hk"), ("wq4_tree_attention.cu", "if (!w.begin(scan, tid, kThreads)) return;"),
    ("wq4_attention_tiles.cu", "bool work = w.begin(scan, tid, kThreads);"), ("wq4_verify.cu", "const int s0 = a.starts[b], s1 = a.starts[b + 1];")])
def test_a_read_moved_ahead_is_seen(name, read):
    """The wait of each kernel moved behind the statement that follows it."""
    text = code(name)
    assert read in text
    late = text.replace(WAIT + ' ::: "memory");', "").replace(read, read + " const float x = a.inv_freq[0]; " + WAIT + ' ::: "memory");' if name == "wq4_append.cu"
                                                              else read + " " + WAIT + ' ::: "memory");')
    assert any(TOUCHES.search(p) for p in ahead_of_the_wait(late))
