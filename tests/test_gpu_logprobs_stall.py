"""Log probabilities: the wait of a cluster's join runs out, is reported, and the next call is right; and what the binding refuses."""
import pytest
import torch

from tests.test_gpu_logprobs import check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,V", [(1, 131072), (5, 70001), (70, 20000)])
def test_a_wait_that_runs_out_is_reported(lib, T, V, dtype):
    x = make(T, V, dtype, 1)
    lib.set_option(lib.OPT_TIMEOUT_CYCLES, 2000000)
    lib.set_option(lib.OPT_TEST_STALL, 1)
    try:
        lib.token_logprobs(x, top_k=4)
        assert lib.get_last_error() == lib.ERR_TIMEOUT
    finally:
        lib.set_option(lib.OPT_TEST_STALL, 0)
        lib.set_option(lib.OPT_TIMEOUT_CYCLES, 0)
    check(lib, x, 4)


def test_rows_without_a_wait_do_not_stall(lib):
    """A CTA that has its row to itself waits for nothing (as the norm and the gated activation)."""
    x = make(400, 3000, "bf16", 2)
    want = lib.token_logprobs(x, top_k=3)
    q, s = lib.silu_mul_quant(x)
    lib.set_option(lib.OPT_TEST_STALL, 1)
    try:
        got = lib.token_logprobs(x, top_k=3)
        q2, s2 = lib.silu_mul_quant(x)
    finally:
        lib.set_option(lib.OPT_TEST_STALL, 0)
    assert lib.get_last_error() == 0
    assert all(torch.equal(a, b) for a, b in zip(got[1:], want[1:]))
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)
