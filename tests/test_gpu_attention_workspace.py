"""A call without a workspace of the caller's: what is cleared for it, and that what memory holds does not matter."""
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
