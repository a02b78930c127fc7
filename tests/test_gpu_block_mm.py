"""The block-scaled 8-bit product against the fp64 oracle.

Tolerance of an element: the tensor core adds a block's 128 products in fp32 (each addition within
2^-22 of the sum of magnitudes, as measured), the blocks' parts are added in fp32 with one rounding each
and a scale factor of one rounding; with at most 128 blocks 2^-16 of the sum of the terms' magnitudes
bounds it with room, plus half a step of the output type."""
import numpy as np
import pytest
import torch

from oracle import rows_oracle as R

pytestmark = pytest.mark.gpu
BITS = {torch.bfloat16: 8, torch.float16: 11, torch.float32: 24}


def operand(rows, K, seed, nan_at=None):
    """e4m3 codes with a padded row stride, values over the format's whole range."""
    rng = np.random.default_rng(seed)
    v = rng.normal(size=(rows, K)) * 2.0 ** rng.integers(-4, 6, size=(rows, 1))
    codes = np.zeros((rows, (K + 15) // 16 * 16 + 16), dtype=np.uint8)
    codes[:, :K] = R.encode_e4m3(np.clip(v, -448, 448))
    codes[:, K:] = 0x7f                                # NaN: must not be read
    if nan_at:
        codes[nan_at] = 0x7f
    t = torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn)[:, :K]
    return codes[:, :K], t


def scale_rows(blocks, n, seed, pad):
    rng = np.random.default_rng(seed)
    s = np.full((blocks, pad), np.nan, dtype=np.float32)
    s[:, :n] = np.exp(rng.normal(size=(blocks, n))) * 0.01
    return s[:, :n], torch.from_numpy(s).cuda()[:, :n]


def check(lib, M, N, K, dtype, seed=0, out=None):
    kb, nb = -(-K // 128), -(-N // 128)
    xq, x = operand(M, K, seed)
    wq, w = operand(N, K, seed + 1)
    sx, dsx = scale_rows(kb, M, seed + 2, (M + 3) // 4 * 4 + 4)
    sw, dsw = scale_rows(nb, kb, seed + 3, kb + 3)
    y = lib.block_mm(x, dsx, w, dsw, out=out, dtype=None if out is not None else dtype)
    assert lib.get_last_error() == 0
    want, mag = R.block_mm(xq, sx, wq, sw)
    got = y.double().cpu().numpy()
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(want), 2.0 ** -126))) - BITS[dtype] + 1)
    if dtype == torch.float16:
        assert np.abs(want).max() < 60000
        step = np.maximum(step, 2.0 ** -24)
    bad = np.abs(got - want) > 2.0 ** -16 * mag + 0.5 * step * (1 + 2.0 ** -8)
    assert not bad.any(), (M, N, K, np.argwhere(bad)[:5], int(bad.sum()))
    return y


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 32, 33, 64, 65, 128, 129, 300])
@pytest.mark.parametrize("N,K", [(1, 16), (7, 128), (128, 112), (129, 144), (256, 640), (300, 2064)])
def test_ragged_sizes(lib, M, N, K):
    check(lib, M, N, K, torch.float32, seed=M + N)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (16, 1000, 4096), (48, 520, 1024), (100, 4100, 272), (333, 700, 2064),
                                   (1300, 2100, 272), (2048, 2560, 512), (700, 14336, 144)])
def test_output_types(lib, M, N, K, dtype):
    check(lib, M, N, K, dtype, seed=7)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M", [1, 7, 16, 50, 95])
@pytest.mark.parametrize("N,K", [(128, 1024), (2300, 1040), (2440, 900), (3000, 1536), (3700, 656), (5000, 400), (6000, 640), (2560, 1536), (2000, 896)])
def test_tiles_shared_by_clusters_of_every_size(lib, M, N, K, dtype):
    """1 to 47 tiles, each cut along K for 8 CTAs down to 2."""
    check(lib, M, N, K // 16 * 16, dtype, seed=M)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("offset,pad", [(0, 3), (1, 8), (8, 8)])
@pytest.mark.parametrize("M,N", [(5, 200), (90, 333), (2100, 2300)])
def test_strided_output_and_untouched_padding(lib, M, N, offset, pad, dtype):
    big = torch.full((M + 1, N + offset + pad), 9.0, dtype=dtype, device="cuda")
    check(lib, M, N, 256, dtype, seed=3, out=big[:M, offset:offset + N])
    assert bool((big[:, :offset] == 9).all()) and bool((big[:, offset + N:] == 9).all()) and bool((big[M] == 9).all())


@pytest.mark.parametrize("M,N,K", [(8, 14336, 4096), (257, 1024, 4096), (1024, 4096, 1024)])
def test_identical_from_run_to_run(lib, M, N, K):
    first = check(lib, M, N, K, torch.float32, seed=5)
    again = check(lib, M, N, K, torch.float32, seed=5)
    assert torch.equal(first, again)


@pytest.mark.parametrize("M,N", [(9, 300), (70, 300), (1500, 2600)])
def test_nan_stays_in_its_row_and_column(lib, M, N):
    K = 384
    _, x = operand(M, K, 1, nan_at=(M // 2, 200))
    _, w = operand(N, K, 2, nan_at=(N - 1, 383))
    _, sx = scale_rows(3, M, 3, (M + 3) // 4 * 4)
    _, sw = scale_rows(-(-N // 128), 3, 4, 4)
    nan = torch.isnan(lib.block_mm(x, sx, w, sw, dtype=torch.float32)).cpu()
    want = torch.zeros(M, N, dtype=torch.bool)
    want[M // 2] = True
    want[:, N - 1] = True
    assert lib.get_last_error() == 0 and torch.equal(nan, want)


def test_no_tokens(lib):
    _, w = operand(64, 128, 1)
    _, sw = scale_rows(1, 1, 2, 4)
    q, s = lib.alloc_quant_rows(0, 128)
    assert lib.block_mm(q, s, w, sw).shape == (0, 64) and lib.get_last_error() == 0


@pytest.mark.parametrize("M", [4, 100, 3000])
def test_a_wait_that_runs_out_is_reported(lib, M):
    """Every CTA makes one wait that nothing ends: the call stops early, reports it, and the next one is right."""
    N, K = 2560, 512
    _, x = operand(M, K, 1)
    _, w = operand(N, K, 2)
    _, sx = scale_rows(4, M, 3, (M + 3) // 4 * 4)
    _, sw = scale_rows(20, 4, 4, 4)
    lib.set_option(lib.OPT_TIMEOUT_CYCLES, 2000000)
    lib.set_option(lib.OPT_TEST_STALL, 1)
    try:
        lib.block_mm(x, sx, w, sw)
        assert lib.get_last_error() == lib.ERR_TIMEOUT
    finally:
        lib.set_option(lib.OPT_TEST_STALL, 0)
        lib.set_option(lib.OPT_TIMEOUT_CYCLES, 0)
    check(lib, M, N, K, torch.bfloat16)


@pytest.mark.parametrize("pdl", [0, -1])
def test_a_layer_in_stream_order(lib, pdl):
    """norm -> product -> gated -> product, each reading what the one before wrote, against the fp64
    definitions of the quantised values actually produced."""
    T, D, F = 70, 512, 640
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, D, generator=g, device="cuda").bfloat16()
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    w1q, w1 = operand(2 * F, D, 2)
    w2q, w2 = operand(D, F, 3)
    s1, ds1 = scale_rows(10, 4, 4, 4)
    s2, ds2 = scale_rows(4, 5, 5, 8)
    lib.set_option(lib.OPT_PDL, pdl)
    try:
        for _ in range(3):
            q, s, _ = lib.add_rmsnorm_quant(x, w)
            gu = lib.block_mm(q, s, w1, ds1)
            q2, sc2 = lib.silu_mul_quant(gu)
            out = lib.block_mm(q2, sc2, w2, ds2, dtype=torch.float32)
    finally:
        lib.set_option(lib.OPT_PDL, 0)
    assert lib.get_last_error() == 0
    codes = lambda t: t.contiguous().view(torch.uint8).cpu().numpy()   # noqa: E731
    y1, m1 = R.block_mm(codes(q), s.cpu().numpy(), w1q, s1)
    assert np.all(np.abs(gu.double().cpu().numpy() - y1) <= 2.0 ** -16 * m1 + 2.0 ** -8 * np.abs(y1))
    y2, m2 = R.block_mm(codes(q2), sc2.cpu().numpy(), w2q, s2)
    assert np.all(np.abs(out.double().cpu().numpy() - y2) <= 2.0 ** -16 * m2 + 2.0 ** -23 * np.abs(y2))


@pytest.mark.parametrize("M,N,K", [(3, 300, 400), (20, 520, 1040), (60, 14336, 128), (200, 300, 2064), (1300, 2100, 272)])
def test_under_the_bounds_checks(lib, M, N, K):
    """Every form of the kernel in the bounds-checking build: right, and no check fires."""
    lib.build(debug=True)
    old = lib.use_library(lib.DEBUG_LIB_PATH)
    try:
        check(lib, M, N, K, torch.bfloat16, seed=9)
        assert lib.last_violation() is None
    finally:
        lib.restore_library(old)
