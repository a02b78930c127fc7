"""Decisions on drafts next to their borders, where the sum over the vocabulary has to be right to many bits.

The weights of these rows are 1 and w = exp(-15.3125), 2^-22.1: to fp32, a sum of a few ones is the same with such a w and without. The sum
of N1 ones and N2 w is held by a pair of floats to 2^-44, and the kernel's w is within 2 ulp of the exponential, 2^-22 of it: N2 w is
2^-19 of the sum, so 1 / sum is known to 2^-40 of it, and random numbers of 24 bits lie on one side of it or the other."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
LOW = -15.3125


def rows(V, ones, count):
    """[count][V] bf16 logits: 0 in the first `ones` columns of each eighth, LOW elsewhere."""
    x = torch.full((8, V // 8), LOW, device="cuda")
    x[:, :ones] = 0.0
    return x.view(1, V).to(torch.bfloat16).expand(count, V).contiguous()


def decide(lib, logits, u, draft=0):
    """Whether each pair of rows keeps the draft, with a random number each."""
    B = len(u)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")   # noqa: E731
    uniforms = torch.zeros(2 * B, device="cuda")
    uniforms[1::2] = torch.tensor(u, dtype=torch.float32)
    out = lib.verify_drafts(logits[:2 * B], torch.full((2 * B,), draft, device="cuda"), ints([-1, 0] * B), ints(list(range(0, 2 * B + 1, 2))),
                            uniforms, torch.full((B,), 0.5, device="cuda"), 2)
    assert lib.get_last_error() == 0
    return out[0].tolist()


@pytest.mark.parametrize("V,ones", [(262144, 4096), (131072, 1024), (32768, 256)])
def test_a_first_draft_on_the_border(lib, V, ones):
    total = 8 * ones + (V - 8 * ones) * float(np.exp(LOW))
    border = 1.0 / total
    near = np.float32(border)
    u = [near]
    for _ in range(24):
        u = [np.nextafter(u[0], np.float32(0))] + u + [np.nextafter(u[-1], np.float32(1))]
    u += [np.float32(1 / (8 * ones))]
    want = [int(float(x) < border) for x in u]
    assert 0 < sum(want) < len(want) and min(abs(float(x) * total - 1) for x in u) > 2.0 ** -36
    logits = rows(V, ones, 2 * 192)
    assert decide(lib, logits, u) == want
    # alone, in a small batch, in a large one: other numbers of threads and CTAs, the same decisions
    assert [decide(lib, logits, [x])[0] for x in u[::3]] == want[::3]
    many = (u * 4)[:192]
    assert decide(lib, logits, many) == (want * 4)[:192]
