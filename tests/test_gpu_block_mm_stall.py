"""The block-scaled product cut along K over clusters of every size: when a wait runs out the call reports it after every
part on its way has landed, calls behind it are right, and so they are time and again."""
import pytest
import torch

from tests.test_gpu_block_mm import check, operand, scale_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(1, 128, 1024), (16, 2440, 900), (50, 3700, 656), (95, 2300, 1040), (100, 5000, 400), (300, 700, 2064)])
def test_clusters_that_give_up(lib, M, N, K):
    K = K // 16 * 16
    kb, nb = -(-K // 128), -(-N // 128)
    _, x = operand(M, K, 1)
    _, w = operand(N, K, 2)
    _, sx = scale_rows(kb, M, 3, (M + 3) // 4 * 4)
    _, sw = scale_rows(nb, kb, 4, kb)
    for _ in range(3):
        lib.set_option(lib.OPT_TIMEOUT_CYCLES, 200000)
        lib.set_option(lib.OPT_TEST_STALL, 1)
        try:
            lib.block_mm(x, sx, w, sw)
            lib.block_mm(x, sx, w, sw)                       # behind it, and as soon as its CTAs go
            assert lib.get_last_error() == lib.ERR_TIMEOUT
        finally:
            lib.set_option(lib.OPT_TEST_STALL, 0)
            lib.set_option(lib.OPT_TIMEOUT_CYCLES, 0)
        check(lib, M, N, K, torch.bfloat16)
