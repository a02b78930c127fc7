"""Temperatures so small that they and their reciprocals lie at the ends of fp32, with scaled logits that are still finite."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heat", [3e-39, 3.5e-39, 4.1e-39, 5e-39, 1e-38])
@pytest.mark.parametrize("V", [40, 50000, 400000])
def test_temperatures_next_to_the_least(lib, heat, V):
    """Tied largest logits share p; a draft among them is kept by its share, one that is not is not."""
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")   # noqa: E731
    x = torch.full((8, V), -float("inf"), device="cuda")
    x[:, [3, V // 2, V - 1]] = 0.25                  # 0.25 / heat is finite; p: a third each
    x[4:, 7] = 0.125                                 # (and nothing beside those)
    tokens = torch.tensor([0, V // 2, 0, V // 2, 0, 7, 0, V - 1], device="cuda")
    u = torch.tensor([0, 0.33, 0, 0.34, 0, 0.0, 0, 0.2], device="cuda")
    out = lib.verify_drafts(x, tokens, ints([-1, 0] * 4), ints([0, 2, 4, 6, 8]), u, torch.full((4,), 0.4, device="cuda"), 2,
                            temperature=torch.full((4,), heat, device="cuda"))
    assert lib.get_last_error() == 0
    assert out[0].tolist() == [1, 0, 0, 1]
    # (a draft that is not kept leaves two thirds: 0.4 of them lies in the first)
    assert out[2].tolist() == [V // 2, 3, V // 2, V // 2]
