"""RMS norm and gated activation into 8-bit rows against the fp64 oracle.

Tolerances. y is computed in fp32: the sum of squares adds at most 32 terms per thread and 10 across the
CTA, so its relative error is below 42 x 2^-24, halved by the root; the rest is a handful of roundings
(and for the gated form exp2 and a division of 2 ulp each): 2^-18 bounds y's relative error with
room, and a scale's. A code is the nearest one to y / s up to that error: half an e4m3 step plus 2^-17 of
the value. 16-bit outputs are within half a step of theirs, up to the same error."""
import numpy as np
import pytest
import torch

from oracle import rows_oracle as R

pytestmark = pytest.mark.gpu
REL = 2.0 ** -18
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def host(t):
    return t.detach().double().cpu().numpy()


def check_quantised(q, scales, y, rel=REL):
    codes = q.contiguous().view(torch.uint8).cpu().numpy()
    s = host(scales)
    want = R.block_scales(y)
    assert np.all(np.abs(s - want) <= rel * want)
    v = y / R.spread(s, y.shape[1])
    got = R.decode_e4m3(codes)
    assert np.all(np.abs(got - v) <= 0.5 * R.e4m3_step(np.minimum(np.abs(v), 448)) + 2 * rel * np.abs(v))


def check_half(got, want, dtype, rel=REL):
    bits = 8 if dtype == "bf16" else 11
    g = host(got)
    tiny = 2.0 ** -24 if dtype == "fp16" else 0.0
    step = np.maximum(2.0 ** (np.floor(np.log2(np.maximum(np.abs(want), 1e-300))) - bits + 1), tiny)
    assert np.all(np.abs(g - want) <= 0.5 * step * (1 + 2.0 ** -10) + rel * np.abs(want))


def make(T, D, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(T, D, generator=g, device="cuda") * scale).to(TYPES[dtype])


SIZES = [(1, 1), (3, 7), (2, 8), (5, 120), (1, 128), (4, 129), (7, 136), (1, 4096), (33, 2064), (3, 4100), (2, 8192),
         (3, 8200), (2, 16384), (1, 16385), (2, 32768), (300, 512),
         # more rows than the SMs hold at once: a warp per row, two and four vectors per thread
         (613, 1), (700, 250), (641, 507), (620, 4104), (611, 5003), (609, 8193), (609, 16380)]


@pytest.mark.parametrize("T,D", SIZES)
@pytest.mark.parametrize("dtype,residual", [("bf16", True), ("fp16", False), ("fp16", True)])
def test_norm(lib, T, D, dtype, residual):
    x, r = make(T, D, dtype, 1), make(T, D, dtype, 2, 4.0) if residual else None
    w = make(1, D, dtype, 3)[0]
    y16 = torch.empty_like(x)
    q, s, h = lib.add_rmsnorm_quant(x, w, residual=r, eps=1e-5, y=y16)
    assert lib.get_last_error() == 0
    hh, y = R.add_rmsnorm(host(x), host(w), host(r) if residual else None, 1e-5)
    check_quantised(q, s, y)
    check_half(y16, y, dtype)
    if residual:
        check_half(h, hh, dtype, rel=2.0 ** -24)
    else:
        assert h is None


@pytest.mark.parametrize("T,D", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_gated(lib, T, D, dtype):
    x = make(T, 2 * D, dtype, 4, 3.0)
    q, s = lib.silu_mul_quant(x)
    assert lib.get_last_error() == 0
    check_quantised(q, s, R.silu_mul(host(x)))


@pytest.mark.parametrize("T,D", [(33, 8), (1000, 1), (2501, 99), (1300, 128), (700, 1920), (500, 1921), (300, 4101), (150, 8193)])
def test_gated_rows_that_share_a_cta(lib, T, D):
    x = make(T, 2 * D, "bf16", 21, 3.0)
    q, s = lib.silu_mul_quant(x)
    assert lib.get_last_error() == 0
    check_quantised(q, s, R.silu_mul(host(x)))


@pytest.mark.parametrize("pad,offset", [(8, 0), (8, 8), (3, 0), (8, 1), (5, 3)])
@pytest.mark.parametrize("op", ["norm", "gated"])
def test_strided_rows_and_untouched_padding(lib, op, pad, offset):
    """Rows inside wider buffers, aligned or not; nothing around the outputs is written."""
    T, D = 6, 392
    width = D if op == "norm" else 2 * D
    base = make(T, width + pad + offset, "bf16", 5)
    x = base[:, offset:offset + width]
    big_q = torch.full((T, 416), 7, dtype=torch.uint8, device="cuda")
    big_s = torch.full((6, 8), -3.0, device="cuda")
    q, s = big_q.view(torch.float8_e4m3fn)[:, :D], big_s[:4, :T]
    if op == "norm":
        w = make(1, D, "bf16", 6)[0]
        big_h = torch.full((T, D + 9), 5.0, dtype=torch.bfloat16, device="cuda")
        r = make(T, D, "bf16", 7)
        lib.add_rmsnorm_quant(x, w, residual=r, eps=0.0, q=q, scales=s, residual_out=big_h[:, 1:D + 1])
        h, y = R.add_rmsnorm(host(x), host(w), host(r), 0.0)
        check_half(big_h[:, 1:D + 1], h, "bf16", rel=2.0 ** -24)
        assert bool((big_h[:, :1] == 5).all()) and bool((big_h[:, D + 1:] == 5).all())
    else:
        lib.silu_mul_quant(x, q=q, scales=s)
        y = R.silu_mul(host(x))
    assert lib.get_last_error() == 0
    check_quantised(q, s, y)
    assert bool((big_q[:, D:] == 7).all())
    assert bool((big_s[:4, T:] == -3).all()) and bool((big_s[4:] == -3).all())


@pytest.mark.parametrize("which", ["x", "residual"])
def test_norm_in_place(lib, which):
    x, r, w = make(9, 1000, "fp16", 8), make(9, 1000, "fp16", 9), make(1, 1000, "fp16", 10)[0]
    q0, s0, h0 = lib.add_rmsnorm_quant(x, w, residual=r)
    q1, s1, h1 = lib.add_rmsnorm_quant(x, w, residual=r, residual_out=x if which == "x" else r)
    assert torch.equal(h0, h1) and torch.equal(q0.view(torch.uint8), q1.view(torch.uint8)) and torch.equal(s0, s1)


@pytest.mark.parametrize("D", [256, 250])
def test_norm_special_rows(lib, D):
    """A row of zeros, of the smallest values, one with an infinity, one with a NaN, one whose squares
    overflow fp32: each stays in its own row."""
    x = make(6, D, "bf16", 11)
    x[0] = 0
    x[1] = 1e-38
    x[2, 5] = float("inf")
    x[3, 200] = float("nan")
    x[4] = 3e38
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    q, s, _ = lib.add_rmsnorm_quant(x, w, eps=1e-5)
    v = q.float().cpu() * torch.repeat_interleave(s.t(), 128, dim=1)[:, :D].cpu()
    assert lib.get_last_error() == 0
    assert bool((v[0] == 0).all()) and bool((s[:, 0].cpu() == 2.0 ** -126).all())
    _, y = R.add_rmsnorm(host(x[[1, 5]]), host(w), None, 1e-5)
    check_quantised(q[[1, 5]], s[:, [1, 5]], y)
    assert bool(torch.isnan(v[2, 5])) and bool((v[2, :5] == 0).all())       # 1 / sqrt(inf) = 0, inf * 0 = NaN
    assert bool(torch.isnan(v[3]).all())                                    # the norm is NaN
    assert bool((v[4] == 0).all())                                          # 1 / sqrt(inf)


def test_gated_special_values(lib):
    inf = float("inf")
    D = 256
    x = make(4, 2 * D, "bf16", 12)
    x[0, :D] = -1000.0                       # silu -> 0
    x[0, D:] = 3e38                          # (and times the largest u still 0)
    x[1, 3], x[1, D + 3] = 1000.0, 1000.0
    x[2, 130] = float("nan")
    x[3, 7], x[3, D + 7] = inf, 1.0
    q, s = lib.silu_mul_quant(x)
    assert lib.get_last_error() == 0
    v = q.float().cpu() * torch.repeat_interleave(s.t(), 128, dim=1).cpu()
    assert bool((v[0] == 0).all())
    assert abs(float(v[1, 3]) - 1e6) <= 1e6 * 2.0 ** -4
    assert bool(torch.isnan(v[2, 130])) and int(torch.isnan(v[2]).sum()) == 1
    assert bool(torch.isnan(v[3, :128]).all()) and not bool(torch.isnan(v[3, 128:]).any())
    check_quantised(q[1:2], s[:, 1:2], R.silu_mul(host(x[1:2])))


def test_empty(lib):
    x = torch.empty(0, 512, dtype=torch.bfloat16, device="cuda")
    q, s, h = lib.add_rmsnorm_quant(x, torch.ones(512, dtype=torch.bfloat16, device="cuda"), residual=x)
    assert q.shape == (0, 512) and s.shape == (4, 0) and h.shape == (0, 512)
    q, s = lib.silu_mul_quant(x)
    assert q.shape == (0, 256) and s.shape == (2, 0)
    assert lib.get_last_error() == 0


def test_side_stream(lib):
    x, w = make(64, 4096, "bf16", 13), make(1, 4096, "bf16", 14)[0]
    want = lib.add_rmsnorm_quant(x, w)[0].view(torch.uint8).cpu()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q = lib.add_rmsnorm_quant(x, w)[0]
    side.synchronize()
    assert torch.equal(q.view(torch.uint8).cpu(), want)
