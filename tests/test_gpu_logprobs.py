"""Log probabilities, entropy and top tokens against the fp64 oracle.

Tolerances. d = x - max is exact to half an ulp; exp2 of d log2(e) errs by 2^-22 + |d| 2^-23, which
weighs d exp(d); sums of V terms add V / 512 terms a thread and a tree over threads, at most 2^-24 each of
the running sum: at V <= 160001 the relative error of the sum is below 2^-15 in the worst case and log z's
absolute error with it; 2e-5 covers every quantity here (log probabilities also by half an ulp of theirs).
The entropy has two such errors and |log z|, |s / z| <= 12: 5e-5. Indices are exact."""
import numpy as np
import pytest
import torch

from oracle import rows_oracle as R

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def make(T, V, dtype, seed, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, V + pad, generator=g, device="cuda") * 3
    return x.to(TYPES[dtype])[:, :V]


def check(lib, x, k, tokens=None):
    T, V = x.shape
    if tokens is None:
        tokens = torch.from_numpy(np.random.default_rng(T + V).integers(0, V, T)).cuda()
    lp, ent, ids, tlp = lib.token_logprobs(x, tokens, top_k=k)
    assert lib.get_last_error() == 0
    wlp, went, wids, wtlp = R.token_logprobs(x.double().cpu().numpy(), tokens.cpu().numpy(), k)

    def near(got, want, tol):
        g = got.double().cpu().numpy()
        same = (g == want) | (np.isnan(g) & np.isnan(want))
        with np.errstate(invalid="ignore"):
            close = np.isfinite(g) & np.isfinite(want) & (np.abs(g - want) <= tol + 2.0 ** -23 * np.abs(want))
        assert (same | close).all(), (np.argwhere(~(same | close))[:5], g[~(same | close)][:5], want[~(same | close)][:5])

    near(lp, wlp, 2e-5)
    near(ent, went, 5e-5)
    if k:
        assert np.array_equal(ids.cpu().numpy(), wids)
        near(tlp, wtlp, 2e-5)
    else:
        assert ids is None and tlp is None


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,V,k", [(1, 1, 1), (3, 2, 2), (2, 7, 0), (5, 8, 8), (4, 9, 5), (3, 31, 20), (7, 64, 32),
                                   (2, 1000, 32), (40, 4097, 5), (1, 8192, 20), (1, 32001, 1), (20, 32001, 32),
                                   (1, 131072, 20), (3, 160001, 20), (80, 20000, 7), (400, 5000, 3)])
def test_sizes(lib, dtype, T, V, k):
    check(lib, make(T, V, dtype, T + V), k)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("pad,offset", [(1, 0), (3, 1), (8, 5), (16, 7)])
def test_rows_off_their_boundaries(lib, dtype, pad, offset):
    x = make(9, 3001 + offset, dtype, 1, pad)[:, offset:]
    check(lib, x, 20)
    x = make(2, 40000 + offset, dtype, 2, pad)[:, offset:]
    check(lib, x, 20)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("V", [50, 6000, 70000])
def test_masked_rows(lib, dtype, V):
    """-inf and the type's lowest value in most places, in all, and in all but fewer than k."""
    low = torch.finfo(TYPES[dtype]).min
    x = make(9, V, dtype, 3)
    keep = torch.rand(V, device="cuda") < 0.1
    x[0, ~keep] = -float("inf")
    x[1, ~keep] = low
    x[2] = -float("inf")
    x[3] = low
    x[4] = -float("inf")
    x[4, V // 2] = 2.0
    x[5] = low
    x[5, [1, V - 1]] = 1.0
    x[6] = -float("inf")
    x[6, V // 3:V // 3 + 9] = -3.0
    x[7, : V - 3] = -float("inf")
    tokens = torch.tensor([0, 0, 0, V - 1, V // 2, 1, V // 3 + 8, V - 1, 5], device="cuda")
    check(lib, x, 20, tokens)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("V", [300, 9000, 70001])
def test_ties_and_orders(lib, dtype, V):
    """All equal, ascending, descending, coarse values, zeros of both signs."""
    x = torch.zeros(6, V, device="cuda")
    x[1] = torch.linspace(-9, 9, V, device="cuda")
    x[2] = torch.linspace(9, -9, V, device="cuda")
    x[3] = torch.randint(0, 3, (V,), device="cuda").float()
    x[4, ::2] = -0.0
    x[5] = -7.0
    x[5, V // 2:] = 7.0
    check(lib, x.to(TYPES[dtype]), 32)


@pytest.mark.parametrize("dtype,stride", [("bf16", 4096), ("fp16", 8), ("fp32", 2048), ("bf16", 32768), ("fp32", 16384)])
def test_the_best_tokens_lie_in_one_threads_share(lib, dtype, stride):
    """The likely tokens sit where one thread (or one warp) of the kernel reads: V / 512 of them above the rest."""
    for T in (1, 30):
        x = make(T, 131072, dtype, 5)
        x[:, 16::stride] += 40.0
        check(lib, x, 32)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_nan_and_inf_rows(lib, dtype):
    x = make(8, 5000, dtype, 6)
    x[1, 7] = float("nan")
    x[2] = float("nan")
    x[3, 4999] = float("inf")
    x[4, 3] = float("nan")
    x[4, 4:] = -float("inf")
    x[5, 100] = float("nan")
    x[5, 200] = float("inf")
    check(lib, x, 4)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("T,V,k", [(330, 50, 20), (700, 50, 32), (330, 4097, 32), (700, 4096, 20), (330, 20001, 5), (700, 20000, 32),
                                   (1300, 1003, 7)])
def test_many_rows_of_every_kind(lib, dtype, T, V, k, pad):
    """As many rows as are taken by fewer threads each: a thread adds V / 128 terms then, below 2e-5 all the same."""
    x = make(T, V, dtype, T + V, pad)
    low = torch.finfo(TYPES[dtype]).min
    x[0::11] = -float("inf")
    x[1::11] = low
    x[2::11, V // 2:] = -float("inf")
    x[3::11, 3:] = low
    x[4::11, 7:] = -float("inf")
    x[5::11] = 0.5
    x[6::11] = torch.linspace(-9, 9, V, device="cuda").to(TYPES[dtype])
    x[7::11] = torch.linspace(9, -9, V, device="cuda").to(TYPES[dtype])
    x[8::11, 16::512] += 40.0
    x[9::11, V // 3] = float("nan")
    check(lib, x, k)


def test_tokens_outside_the_vocabulary(lib):
    x = make(5, 700, "fp32", 7)
    check(lib, x, 1, torch.tensor([-1, 700, 699, 0, -(1 << 40)], device="cuda"))


def test_what_is_asked_for(lib):
    x = make(3, 999, "bf16", 8)
    tok = torch.tensor([1, 2, 3], device="cuda")
    full = lib.token_logprobs(x, tok, top_k=3)
    none = lib.token_logprobs(x, top_k=3)
    assert none[0] is None and all(torch.equal(a, b) for a, b in zip(none[1:], full[1:]))
    bare = lib.token_logprobs(x, tok)
    assert torch.equal(bare[0], full[0]) and bare[2] is None
    assert lib.token_logprobs(x[:0], tok[:0], top_k=2)[2].shape == (0, 2)
    with pytest.raises(ValueError):
        lib.token_logprobs(x, tok.int())
    with pytest.raises(lib.Wq4Error):
        lib.token_logprobs(x, tok, top_k=33)


def test_large_magnitudes(lib):
    """Differences beyond fp32's exponent range, and the widest values of fp32."""
    x = torch.zeros(3, 600, device="cuda")
    x[0, 5], x[0, 6] = 3e38, -3e38
    x[1, :10] = 1e4
    x[2] = torch.linspace(-3e4, 3e4, 600, device="cuda")
    check(lib, x, 12)
