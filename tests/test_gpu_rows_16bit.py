"""RMS norm into 16-bit rows alone, through the C entry point (codes and scales null), against the fp64 oracle with the
tolerances of test_gpu_rows; and the same bits as when codes are asked for too."""
import pytest
import torch

from oracle import rows_oracle as R
from tests.test_gpu_rows import check_half, host, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,D", [(1, 1), (3, 129), (2, 4096), (33, 2064), (2, 16385), (1, 32768), (700, 250), (620, 4104)])
@pytest.mark.parametrize("dtype,residual", [("bf16", True), ("fp16", False)])
def test_norm_writes_16_bit_rows_only(lib, T, D, dtype, residual):
    x, w = make(T, D, dtype, 1), make(1, D, dtype, 2)[0]
    r = make(T, D, dtype, 3, 4.0) if residual else None
    y, h = torch.empty_like(x), torch.empty_like(x) if residual else None
    ptr = lambda t: None if t is None else t.data_ptr()   # noqa: E731
    rc = lib.load_library().wq4_add_rmsnorm_quant(ptr(x), D, ptr(r), D, ptr(w), T, D, 1e-5, lib.DTYPES[dtype], ptr(h), D, ptr(y), D,
                                                  None, 0, None, 0, torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and lib.get_last_error() == 0
    hh, want = R.add_rmsnorm(host(x), host(w), host(r) if residual else None, 1e-5)
    check_half(y, want, dtype)
    if residual:
        check_half(h, hh, dtype, rel=2.0 ** -24)
    both = torch.empty_like(x)
    lib.add_rmsnorm_quant(x, w, residual=r, eps=1e-5, y=both)
    assert torch.equal(both, y)
