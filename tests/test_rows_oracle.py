"""The fp64 oracle of the 8-bit row operators, tied to something other than itself: torch's e4m3
conversion, closed forms, and scale invariants. Runs without a GPU."""
import numpy as np
import pytest
import torch

from oracle import rows_oracle as R


def test_e4m3_values_match_torch():
    codes = np.arange(256, dtype=np.uint8)
    ref = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()
    got = R.decode_e4m3(codes)
    assert np.array_equal(np.isnan(ref), np.isnan(got))
    assert np.array_equal(ref[~np.isnan(ref)], got[~np.isnan(ref)])


def test_e4m3_rounding_matches_torch():
    rng = np.random.default_rng(0)
    pos = R.E4M3[:127]
    v = np.concatenate([rng.normal(size=4000) * 100, rng.normal(size=4000) * 0.02, pos, (pos[1:] + pos[:-1]) / 2, [448.0]])
    v = np.clip(v, -448, 448).astype(np.float32)
    ref = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref, R.encode_e4m3(v.astype(np.float64)))
    assert R.encode_e4m3(np.array([1e6, -1e6])).tolist() == [126, 254]


def test_scales_of_a_block():
    y = np.zeros((2, 200))
    y[1, 130] = -896.0
    y[1, 3] = np.nan
    s = R.block_scales(y)
    assert s.shape == (2, 2)
    assert s[:, 0].tolist() == [R.SCALE_MIN, R.SCALE_MIN] and s[:, 1].tolist() == [R.SCALE_MIN, 2.0]


def test_norm_closed_form():
    h, y = R.add_rmsnorm(np.array([[3.0, -3.0]]), np.array([1.0, 2.0]), np.array([[1.0, -1.0]]), eps=9.0)
    assert h.tolist() == [[4.0, -4.0]] and np.allclose(y, [[0.8, -1.6]])


def test_gated_closed_form():
    y = R.silu_mul(np.array([[0.0, 1000.0, -1000.0, 5.0, 2.0, 3.0]]))
    assert y.tolist() == [[0.0, 2000.0, 0.0]]


def test_product_scales_apply_per_block():
    rng = np.random.default_rng(1)
    xq, wq = rng.integers(0, 126, (3, 256), dtype=np.uint8), rng.integers(0, 126, (130, 256), dtype=np.uint8)
    sx, sw = rng.uniform(0.5, 1, (2, 3)), rng.uniform(0.5, 1, (2, 2))
    y, _ = R.block_mm(xq, sx, wq, sw)
    brute = sum(R.E4M3[xq[2, k]] * sx[k // 128, 2] * R.E4M3[wq[129, k]] * sw[1, k // 128] for k in range(256))
    assert np.isclose(y[2, 129], brute, rtol=1e-12)
    sx[1] *= 2
    y2, _ = R.block_mm(xq, sx, wq, sw)
    one, _ = R.block_mm(xq[:, 128:], sx[1:] / 2, wq[:, 128:], sw[:, 1:])
    assert np.allclose(y2 - y, one)


@pytest.mark.parametrize("V", [2, 10])
def test_logprobs_closed_forms(V):
    x = np.full((4, V), 1.5)
    x[1, 1:] = -np.inf
    x[2] = -np.inf
    x[3] = np.finfo(np.float32).min
    lp, ent, ids, tlp = R.token_logprobs(x, np.array([1, 0, 0, -5]), 2)
    assert np.allclose(lp[:2], [-np.log(V), 0]) and lp[2] == -np.inf and np.isnan(lp[3])
    assert np.allclose(ent, [np.log(V), 0, 0, np.log(V)])
    assert ids.tolist() == [[0, 1], [0, -1], [-1, -1], [0, 1]]
    assert tlp[1, 1] == -np.inf and tlp[2, 0] == -np.inf and np.isclose(tlp[3, 1], -np.log(V))
