"""Log probabilities: a top_k that does not fit 32 bits is refused, not cut to its low bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k", [(1 << 32) + 1, (1 << 32) + 32, 1 << 31, 1 << 40])
def test_a_top_k_beyond_32_bits_is_refused(lib, k):
    with pytest.raises((ValueError, lib.Wq4Error)):
        lib.token_logprobs(torch.zeros(0, 64, device="cuda"), top_k=k)
    assert lib.get_last_error() == 0
