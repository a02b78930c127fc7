"""Log probabilities of rows whose logits are large in magnitude.

Tolerances are those of test_gpu_logprobs_growing: differences of logits are as exact however large the logits
are, half an ulp of the difference."""
import pytest
import torch

from tests.test_gpu_logprobs import TYPES, check
from tests.test_gpu_logprobs_growing import SIZES, growing_and_falling_rows

pytestmark = pytest.mark.gpu
FILLS = [1e3, 3e4, 6.1e4, 1e5, 1e6, 1.1e6, 1e7, 1e8, 1e9, 1e10, 1e20, 1e30, 2e38]


def fills(dtype):
    top = torch.finfo(TYPES[dtype]).max
    return [s * f for f in FILLS if f <= top for s in (1.0, -1.0)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("V", [8, 600, 9000, 70001])
def test_rows_of_one_value(lib, dtype, V):
    f = torch.tensor(fills(dtype), device="cuda")
    check(lib, f[:, None].expand(-1, V).to(TYPES[dtype]).contiguous(), min(5, V))


def masked(V, dtype, seed, rows, keep):
    """A row for each fill value: ordinary logits where keep holds, the fill elsewhere."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    f = torch.tensor(fills(dtype)[:rows], device="cuda")
    x = torch.randn(len(f), V, generator=g, device="cuda") * 3
    return torch.where(keep[None], x, f[:, None].expand(-1, V)).to(TYPES[dtype])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("V,rows", [(600, 40), (20000, 40), (70001, 40), (131072, 2)])
def test_finite_masks(lib, dtype, V, rows):
    """The fill first, last, nearly everywhere, and all over one thread's share of the row."""
    at = torch.arange(V, device="cuda")
    vec = 4 if dtype == "fp32" else 8
    shares = [at // vec % n != 37 for n in (128, 256, 512)]
    for i, keep in enumerate([at >= V // 2, at < V // 2, at == V // 3, (at % 97) == 5, *shares]):
        check(lib, masked(V, dtype, i, rows, keep), 5)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("V", [700, 4097])
def test_finite_masks_of_many_rows(lib, dtype, V):
    """As many rows as are taken by fewer threads each."""
    at = torch.arange(V, device="cuda")
    x = torch.cat([masked(V, dtype, i, 40, keep) for i, keep in enumerate([at >= V // 2, at == V // 3, at >= 0, at < 0])])
    check(lib, x.repeat(700 // len(x) + 1, 1), 5)


@pytest.mark.parametrize("T,V", SIZES)
@pytest.mark.parametrize("lo,hi", [(1e4, 1e5), (1e5, 1e6), (1e6, 1e7), (1e7, 1e9)])
@pytest.mark.parametrize("sign", [1, -1])
def test_growing_and_falling_rows(lib, T, V, lo, hi, sign):
    growing_and_falling_rows(lib, T, V, lo, hi, sign)


def test_differences_of_an_ulp(lib):
    """Neighbouring fp32 values: below 2^23 their differences count, above they are whole numbers."""
    x = torch.full((8, 3000), 1.0, device="cuda")
    for i, c in enumerate([2.0 ** 10, 2.0 ** 17, 2.0 ** 20, 2.0 ** 21, 2.0 ** 22, 2.0 ** 23, 2.0 ** 24, 2.0 ** 30]):
        x[i] = c + torch.arange(3000, device="cuda") % 11 * max(c * 2.0 ** -23, 2.0 ** -4)
    check(lib, x, 12)
    check(lib, -x, 12)
