"""Verification of sequences with more drafts than are held at hand, and the same sequences in small and large batches."""
import numpy as np
import pytest
import torch

from oracle import attention_oracle as A
from tests.test_gpu_verify import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("probs", [False, True])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("counts", [[128, 129, 127], [200, 5, 333]])
def test_many_drafts(lib, probs, tree, counts):
    c = Case(counts, 64, "fp32", probs, tree=tree, seed=counts[0] + tree, spread=2.0)
    c.check(lib)


def test_a_chain_that_is_kept_to_its_end(lib):
    """Every draft is all that the target can say: the walk passes the drafts held at hand."""
    c = Case([400, 130], 50, "fp32", False, tree=False, seed=1)
    c.logits.fill_(-float("inf"))
    rows = torch.arange(len(c.tokens) - 1, device="cuda")
    c.logits[rows, c.tokens[1:]] = 0.0
    c.logits[399, 7], c.logits[529, 9] = 0.0, 0.0
    c.logits[399, c.tokens[400]] = 0.0 if int(c.tokens[400]) == 7 else -float("inf")
    accepted, path, after = c.run(lib)
    assert accepted.tolist() == [399, 129] and after.tolist() == [7, 9]
    assert path[0].tolist() == list(range(1, 400)) and path[1, :129].tolist() == list(range(1, 130))


@pytest.mark.parametrize("V,dtype", [(40001, "bf16"), (131072, "bf16"), (50000, "fp32")])
@pytest.mark.parametrize("probs", [False, True])
def test_alone_and_in_a_batch(lib, V, dtype, probs):
    """Batches set the number of CTAs and threads of a sequence; walks that are not next to a border are the same."""
    c = Case([4] * 100, V, dtype, probs, seed=9, temperature=[0.8, 0.0, 1.2])
    whole = [t.cpu() for t in c.run(lib)]
    n = lambda t: None if t is None else t.cpu().numpy()   # noqa: E731
    compared = 0
    for b in range(0, 100, 7):
        s = slice(4 * b, 4 * b + 4)
        alone = lib.verify_drafts(c.logits[s], c.tokens[s], c.parents[s], torch.tensor([0, 4], dtype=torch.int32, device="cuda"), c.u[s],
                                  c.uf[b:b + 1], 4, draft_probs=None if c.q is None else c.q[s], temperature=c.heat[b:b + 1])
        heat = float(c.heat[b])
        _, p, margin = A.verify(n(c.logits[s].double()), n(c.tokens[s]), n(c.parents[s]), n(c.u[s]), float(c.uf[b]),
                                None if c.q is None else n(c.q[s]), heat)
        if margin <= 2.0 ** -18:                     # (weights may err by 2^-22 here)
            continue
        assert int(alone[0]) == int(whole[0][b]) and alone[1].cpu()[0].tolist() == whole[1][b].tolist()
        upto = np.cumsum(p)
        if np.abs(upto - float(c.uf[b])).min() > 2.0 ** -22:
            assert int(alone[2]) == int(whole[2][b])
            compared += 1
    assert compared >= 6


@pytest.mark.parametrize("probs", [False, True])
def test_the_oracle_compares_nearly_all_walks(probs):
    """What a walk's nearness to a border leaves out of the comparisons of test_gpu_verify."""
    rng = np.random.default_rng(3)
    c = Case(rng.integers(0, 18, 300).tolist(), 300, "fp32", probs, tree=True, seed=4, temperature=[0.7, 0.0, 1.3, 1.0], spread=4.0)
    n = lambda t: None if t is None else t.cpu().numpy()   # noqa: E731
    left_out = 0
    for b in range(300):
        s = slice(c.starts_list[b], c.starts_list[b + 1])
        left_out += A.verify(n(c.logits.double())[s], n(c.tokens)[s], n(c.parents)[s], n(c.u)[s], n(c.uf)[b], None if c.q is None else n(c.q)[s],
                             float(c.heat[b]))[2] <= 1e-4
    assert left_out <= 15
