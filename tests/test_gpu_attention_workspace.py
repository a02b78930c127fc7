"""A call without a workspace of the caller's: what is cleared for it, and that what memory holds does not matter."""
import os
import sys

import pytest
import torch

from tests.test_gpu_tree_attention import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts,D", [([40, 30, 1], 128), ([1, 1, 2], 256), ([3], 64)])
def test_only_the_counters_are_cleared(lib, counts, D, monkeypatch):
    c = Case(counts, [5000, 700, 0][:len(counts)], 8, 2, D, 16, "bf16", True)
    nbytes = lib.tree_attention_workspace_bytes(len(counts), c.most, 8, 2, D)
    want = c.run(lib, workspace=lib.alloc_workspace(nbytes))
    cleared = []
    for name in ("zeros", "zeros_like"):
        real = getattr(torch, name)
        monkeypatch.setattr(torch, name, lambda *a, _real=real, **k: cleared.append(_real(*a, **k)) or cleared[-1])
    zero_ = torch.Tensor.zero_
    monkeypatch.setattr(torch.Tensor, "zero_", lambda t: cleared.append(t) or zero_(t))
    empty = torch.empty                              # memory as another program might have left it
    monkeypatch.setattr(torch, "empty", lambda *a, **k: (lambda t: t.fill_(255) if t.dtype == torch.uint8 else t)(empty(*a, **k)))
    for _ in range(2):
        got = c.run(lib)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert sum(t.numel() * t.element_size() for t in cleared) <= 2 * 4096


def test_the_example_keeps_one_workspace(lib, monkeypatch):
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    try:
        import speculative_decode as E
    finally:
        sys.path.pop(0)
    seen, real = [], lib.tree_attention
    monkeypatch.setattr(lib, "tree_attention", lambda *a, **k: seen.append(k.get("workspace")) or real(*a, **k))
    g = torch.Generator(device="cuda").manual_seed(0)
    model = E.Decoder(256, 2, 512, 2, places=80)
    roots = model.prefill([[1, 2, 3], list(range(40))]).argmax(dim=1)
    for _ in range(2):
        roots = model.step(roots, torch.zeros(2, device="cuda"), g)[1]
    assert lib.get_last_error() == 0
    assert len(seen) == 6 and all(w is not None and w.data_ptr() == seen[0].data_ptr() for w in seen)
