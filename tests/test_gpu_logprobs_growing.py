"""Log probabilities of rows whose maximum grows as they are read.

Tolerances are those of test_gpu_logprobs.check, 2e-5 (entropy 5e-5) and 2^-23 of the value. What they have to
cover: a term is 2^t with t = x log2(e) - R rounded once, an error of 2^-24 |t|, and log2(e) itself to 2^-26;
weighed with 2^t / z, whose mean |t| is at most log2(V) <= 17, that is below 1.2e-6 of z. ex2 errs by 2^-22. What R
leaves out of max log2(e) is taken out of z and s by one further ex2. Each time a thread's maximum grows its sums
are multiplied by an ex2 (2^-22, and 2^-24 for each of two roundings), 2^-21 a move; the later moves outweigh the
earlier, and a thread of 512 or fewer sees at most V / (16 x 128) + 4 <= 14 of them: 7e-6. The sums themselves: V /
256 terms in each half of a thread's sum (V / 1024 with 512 threads), 2^-24 each of the running sum: below 5e-6.
Together below 2e-5. The entropy is log z and a quotient s / z of magnitude at most 12 with such errors in both, of
the same sign where they come from the factors: 5e-5."""
import numpy as np
import pytest
import torch

from tests.test_gpu_logprobs import check

pytestmark = pytest.mark.gpu
SIZES = [(1, 20000), (40, 20000), (300, 60000), (700, 4096), (1216, 20000)]


def compare(got, x, tokens, k):
    """As test_gpu_logprobs.check, of results that are there."""
    class There:
        token_logprobs = staticmethod(lambda *a, **b: got)
        get_last_error = staticmethod(lambda: 0)
    check(There, x, k, tokens)


def growing_and_falling_rows(lib, T, V, lo, hi, sign):
    """Logits that rise (a thread's maximum grows with all it reads), fall, and rise again and again, around centres of every
    magnitude. Rows of a call beyond the first sixteen repeat them, and so must their results."""
    g = torch.Generator().manual_seed(V + int(lo))
    ramp = torch.linspace(0, 1, V, dtype=torch.float64)
    saw = (torch.arange(V) * 37 % 1009).double() / 1009
    rows = []
    for i in range(min(T, 16)):
        c = sign * lo * (hi / lo) ** float(torch.rand((), generator=g))
        span = max(3.0 * (1 + i // 4), abs(c) * 2.0 ** -20)    # (some tens of values near 1e9)
        rows.append(c + span * [ramp, ramp * 4, saw, ramp.flip(0)][i % 4])
    x = torch.stack(rows).float().cuda()
    n = len(x)
    tokens = torch.arange(T, device="cuda") % n * 7
    out = lib.token_logprobs(x.repeat(-(-T // n), 1)[:T].contiguous(), tokens, top_k=7)
    assert lib.get_last_error() == 0
    for o in out:
        assert torch.equal(o, o[:n].repeat(-(-T // n), *[1] * (o.dim() - 1))[:T])
    compare([o[:n] for o in out], x, tokens[:n], 7)


@pytest.mark.parametrize("T,V", SIZES)
@pytest.mark.parametrize("lo,hi", [(10, 100), (100, 1000), (1000, 1e4)])
@pytest.mark.parametrize("sign", [1, -1])
def test_around_ordinary_values(lib, T, V, lo, hi, sign):
    growing_and_falling_rows(lib, T, V, lo, hi, sign)


@pytest.mark.parametrize("T,V", [(1, 70000), (40, 20000), (300, 60000), (1216, 20000)])
@pytest.mark.parametrize("centre", [20.0, 200.0, 700.0, 1500.0, 2800.0, 5000.0, 9000.0, -300.0, -2800.0, -9000.0])
def test_a_maximum_that_moves_late(lib, T, V, centre):
    """Most of a row is a, the rest b a little above it: all that a thread has added up moves to another reference near the
    row's end. a and b are those near `centre` whose references, m log2(e) in fp32, are rounded most differently."""
    m = np.float32(centre) + np.arange(4000, dtype=np.float32) * np.float32(1e-4)
    exact = m.astype(np.float64) * np.log2(np.e)
    r = exact - (m * np.float32(np.log2(np.e))).astype(np.float64)
    half = len(m) // 2
    rows = []
    for sign in (1, -1):
        a, b = m[:half][np.argmax(sign * r[:half])], m[half:][np.argmin(sign * r[half:])]
        for share in (0.5, 0.75, 0.9):
            x = torch.full((V,), float(a), device="cuda")
            x[int(V * share):] = float(b)
            rows.append(x)
    x = torch.stack(rows).repeat(-(-T // 6), 1)
    tokens = torch.arange(len(x), device="cuda") * 0
    out = lib.token_logprobs(x, tokens, top_k=3)
    assert lib.get_last_error() == 0
    compare([o[:6] for o in out], x[:6], tokens[:6], 3)
