"""The scale and the codes of quantised rows, bit for bit.

With g = 64 the gated activation's 1 + exp(-g) is 1 in fp32, so y = 64 u exactly (u has at most 11 significant bits), and the host
knows y: the scale is then max(max |y| / 448, 2^-126) and the codes are y / scale, each quotient rounded to the nearest fp32 and
the codes to the nearest e4m3. No tolerance."""
import numpy as np
import pytest
import torch

from oracle import rows_oracle as R

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def expect(y):
    """(codes, scales [blocks][T]) of fp32 y, with fp32 divisions."""
    T, D = y.shape
    nb = -(-D // 128)
    s = np.empty((nb, T), dtype=np.float32)
    q = np.empty((T, D), dtype=np.uint8)
    with np.errstate(all="ignore"):
        for b in range(nb):
            part = y[:, b * 128:(b + 1) * 128]
            top = np.where(np.isnan(part), np.float32(0), np.abs(part)).max(axis=1)
            s[b] = np.maximum(top / np.float32(448), np.float32(2.0 ** -126))
            q[:, b * 128:(b + 1) * 128] = R.encode_e4m3((part / s[b][:, None]).astype(np.float64))
    return q, s


def check(lib, u):
    T, D = u.shape
    x = torch.cat([torch.full_like(u, 64.0), u], dim=1)
    q, s = lib.silu_mul_quant(x)
    assert lib.get_last_error() == 0
    with np.errstate(over="ignore"):
        y = u.float().cpu().numpy() * np.float32(64)
    want_q, want_s = expect(y)
    assert np.array_equal(s.cpu().numpy(), want_s)
    got = q.contiguous().view(torch.uint8).cpu().numpy()
    got = np.where(got & 127 == 127, 127, got)                   # (a NaN code's sign says nothing)
    want_q = np.where(want_q & 127 == 127, 127, want_q)
    assert np.array_equal(got, want_q), np.argwhere(got != want_q)[:5]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,D", [(2, 5), (900, 128), (600, 4099), (300, 14336)])
def test_exact_scales_and_codes(lib, T, D, dtype):
    g = torch.Generator(device="cuda").manual_seed(T)
    u = torch.randn(T, D, generator=g, device="cuda") * torch.exp(2 * torch.randn(T, 1, generator=g, device="cuda"))
    check(lib, u.to(TYPES[dtype]))


@pytest.mark.parametrize("D", [128, 1000, 4096])
def test_over_the_exponents(lib, D):
    """Rows of every magnitude that bf16 has: the least scale, small and large ones, and the largest that does not overflow."""
    g = torch.Generator(device="cuda").manual_seed(D)
    e = torch.linspace(-132, 119, 700, device="cuda").floor()[:, None]
    u = (torch.randn(700, D, generator=g, device="cuda").clamp(-3.5, 3.5).double() * 2.0 ** e.double()).bfloat16()
    check(lib, u)


def test_ties(lib):
    """Quotients that lie on the boundary between two codes (448 as the largest: the scale is a power of two)."""
    pos = torch.from_numpy(R.E4M3[:127].copy()).cuda()
    v = torch.cat([pos, (pos[1:] + pos[:-1]) / 2])
    v = torch.cat([v, -v])
    rows = []
    for shift in (-120, -60, 0, 3, 90):
        for i in range(0, len(v), 127):
            rows.append(torch.cat([torch.tensor([448.0], device="cuda", dtype=torch.float64), torch.nn.functional.pad(v[i:i + 127], (0, max(0, 127 - len(v[i:i + 127]))))]) * 2.0 ** shift)
    check(lib, torch.stack(rows).bfloat16())


def test_special_blocks(lib):
    u = torch.randn(6, 300, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").bfloat16()
    u[0, 3] = float("nan")
    u[1, 200] = float("inf")
    u[2, 130] = -float("inf")
    u[2, 131] = float("nan")
    u[3] = 0
    u[4, :128] = float("nan")
    u[5, 7] = 1e38                                               # 64 u overflows
    check(lib, u)
