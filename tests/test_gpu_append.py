"""Keys and values into a paged cache, with norms and rotation, against the fp64 oracle.

Tolerance. A result is rounded once, by half a step of its type (eps / 2 of it). Ahead of that, in fp32 (u = 2^-24): mean of
squares, rsqrt (2 ulp) and two products err by less than 12 u of a feature; the angle's fraction of a turn is held to 2^-25
turns, 2 pi 2^-25 = 3.2 u rad, and cos and sin to 2 u; two products and a sum add 3 u. In all less than 24 u of |a| + |b|
of the pair."""
import numpy as np
import pytest
import torch

from oracle import attention_oracle as A

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def make(T, Hq, Hk, D, R, dtype, norm, page, seed=0, far=131072):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = TYPES[dtype]
    rows = torch.randn(T, Hq + 2 * Hk, D, generator=g, device="cuda").to(dt)
    pages = -(-T // page) + 2
    k_cache, v_cache = (torch.randn(pages, page, Hk, D, generator=g, device="cuda").to(dt) for _ in "kv")
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T]
    pos = torch.randint(0, far, (T,), generator=g, device="cuda")
    freq = (1e4 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / max(R, 1))).float() if R else None
    w = [(1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(dt) if norm else None for _ in "qk"]
    return rows, k_cache, v_cache, slots, pos if R else None, freq, w


def near(got, want, a, b, dtype):
    """|got - want| within half a step and 24 2^-24 (|a| + |b|), a and b a pair's features (their sizes)."""
    g = f64(got)
    eps = torch.finfo(TYPES[dtype]).eps
    tol = eps / 2 * np.abs(want) * (1 + eps) + 24 * 2.0 ** -24 * (a + b) + torch.finfo(TYPES[dtype]).tiny * eps
    assert (np.abs(g - want) <= tol).all(), np.abs(g - want).max()


def check(lib, T, Hq, Hk, D, R, dtype, norm, interleaved, page, rows=None, in_place=False, far=131072, seed=0):
    made, k_cache, v_cache, slots, pos, freq, (qw, kw) = make(T, Hq, Hk, D, R, dtype, norm, page, seed, far)
    rows = made if rows is None else rows
    q, k, v = (rows[:, :Hq] if Hq else None), rows[:, Hq:Hq + Hk], rows[:, Hq + Hk:]
    n = (lambda t: None if t is None else t.cpu().numpy())
    args = (f64(q), f64(k), f64(v), f64(k_cache), f64(v_cache), n(slots), n(pos), f64(freq), f64(qw if Hq else None), f64(kw), 1e-6, interleaved)
    want_q, want_k, want_v = A.rope_append(*args)
    # the sizes of the features ahead of the rotation, each with its partner's
    flat = A.rope_append(*args[:6], None, None, *args[8:])
    idx = np.arange(D)
    if R:
        idx[:R] = idx[:R] ^ 1 if interleaved else np.concatenate([idx[R // 2:R], idx[:R // 2]])
    out = lib.rope_append(q, k, v, k_cache, v_cache, slots, pos, freq, q_weight=qw if Hq else None, k_weight=kw, eps=1e-6,
                          interleaved=interleaved, q_out=q if in_place else None)
    assert lib.get_last_error() == 0
    if Hq:
        near(out, want_q, np.abs(flat[0]), np.abs(flat[0][..., idx]), dtype)
    near(k_cache, want_k, np.abs(flat[1]), np.abs(flat[1][..., idx]), dtype)
    assert np.array_equal(f64(v_cache), want_v)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,R,norm,page", [(1, 32, 8, 128, 128, True, 16), (7, 4, 1, 64, 64, False, 48), (3, 14, 2, 80, 32, True, 16),
                                                    (5, 3, 3, 192, 64, True, 1), (2, 2, 1, 256, 256, True, 7), (19, 1, 1, 16, 16, True, 3),
                                                    (2, 70, 9, 512, 128, False, 5), (4, 2, 2, 96, 0, True, 16), (6, 8, 4, 64, 16, False, 32)])
def test_heads(lib, dtype, interleaved, T, Hq, Hk, D, R, norm, page):
    check(lib, T, Hq, Hk, D, R, dtype, norm, interleaved, page)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,R", [(3, 2, 1, 1, 0), (3, 2, 1, 2, 2), (5, 3, 2, 65, 30), (2, 2, 1, 72, 24), (2, 1, 1, 1024, 1024), (4, 5, 1, 100, 10)])
def test_odd_heads(lib, dtype, interleaved, T, Hq, Hk, D, R):
    check(lib, T, Hq, Hk, D, R, dtype, True, interleaved, 5)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("D,offset", [(64, 0), (64, 1), (66, 0)])
def test_strided_rows_and_in_place(lib, in_place, D, offset):
    """Heads ahead of tokens, rows off their boundaries, queries written where they were read."""
    T, Hq, Hk = 9, 4, 2
    base = torch.randn(Hq + 2 * Hk, T, D + 8, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)).bfloat16()
    rows = base[:, :, offset:offset + D].transpose(0, 1)
    check(lib, T, Hq, Hk, D, 32, "bf16", True, False, 16, rows=rows, in_place=in_place)


@pytest.mark.parametrize("T", [0, 1, 2, 513, 3001])
def test_token_counts(lib, T):
    check(lib, T, 2, 1, 64, 64, "bf16", True, False, 64)


def test_keys_and_values_alone(lib):
    check(lib, 11, 0, 4, 128, 128, "bf16", True, False, 16)


def test_far_positions(lib):
    """Positions up to 2^40, and below zero: the angle is the exact product's."""
    made, k_cache, v_cache, slots, pos, freq, _ = make(6, 1, 1, 64, 64, "fp16", False, 16)
    pos = torch.tensor([0, -5, 2 ** 24 + 1, 10 ** 9 + 7, 2 ** 40 + 12345, -2 ** 33], device="cuda")
    q, k, v = made[:, :1], made[:, 1:2], made[:, 2:]
    out = lib.rope_append(q, k, v, k_cache, v_cache, slots, pos, freq)
    from fractions import Fraction
    pi = Fraction(314159265358979323846264338327950288419716939937510582097494459, 10 ** 62)
    x = f64(q)[:, 0]
    for t, p in enumerate(pos.tolist()):
        w = np.array([float(Fraction(p) * Fraction(float(f)) % (2 * pi)) for f in freq.cpu()])
        want = np.concatenate([x[t, :32] * np.cos(w) - x[t, 32:] * np.sin(w), x[t, 32:] * np.cos(w) + x[t, :32] * np.sin(w)])
        size = np.tile(np.abs(x[t, :32]) + np.abs(x[t, 32:]), 2)
        assert (np.abs(f64(out)[t, 0] - want) <= 2.0 ** -11 * np.abs(want) * 1.001 + 24 * 2.0 ** -24 * size + 2.0 ** -25).all()


def test_padded_tokens_and_slots_outside(lib):
    """A negative slot leaves the cache alone; one beyond it too, and is reported. Every query is written."""
    rows, k_cache, v_cache, slots, pos, freq, _ = make(40, 2, 1, 64, 64, "bf16", False, 16)
    before = k_cache.clone(), v_cache.clone()
    slots = torch.full((40,), -1, device="cuda", dtype=torch.int64)
    slots[3] = -2 ** 40
    args = (rows[:, :2], rows[:, 2:3], rows[:, 3:], k_cache, v_cache)
    out = lib.rope_append(*args, slots, pos, freq)
    assert lib.get_last_error() == 0
    assert torch.equal(k_cache, before[0]) and torch.equal(v_cache, before[1])
    slots[5] = k_cache.shape[0] * 16
    slots[6] = 2 ** 33
    for D in (64, 62):                               # both kernels
        cut = [x[..., :D] for x in args]
        lib.rope_append(*cut, slots, pos, freq[:D // 2].contiguous())
        assert lib.get_last_error() == lib.ERR_INVALID
        assert torch.equal(k_cache, before[0]) and torch.equal(v_cache, before[1])
    assert torch.equal(out, lib.rope_append(*args, torch.arange(40, device="cuda"), pos, freq))


def test_nan_and_infinity_stay_in_their_head(lib):
    rows, k_cache, v_cache, slots, pos, freq, (qw, kw) = make(4, 2, 1, 64, 64, "bf16", True, 16)
    rows[1, 0, 5] = float("nan")
    rows[2, 2, 7] = float("inf")
    rows[3, 3, 1] = float("-inf")
    out = lib.rope_append(rows[:, :2], rows[:, 2:3], rows[:, 3:], k_cache, v_cache, slots, pos, freq, qw, kw)
    bad = ~torch.isfinite(out).all(dim=2).cpu()
    assert bad.nonzero().tolist() == [[1, 0]]
    flat = k_cache.view(-1, 64)[slots]
    assert (~torch.isfinite(flat).all(dim=1)).nonzero().flatten().tolist() == [2]
    assert v_cache.view(-1, 64)[slots][3, 1] == -float("inf")


def test_captured_and_replayed_on_another_stream(lib):
    rows, k_cache, v_cache, slots, pos, freq, (qw, kw) = make(33, 4, 2, 128, 128, "bf16", True, 16)
    q, k, v = rows[:, :4], rows[:, 4:6], rows[:, 6:]
    out = torch.empty_like(q, memory_format=torch.contiguous_format)
    lib.rope_append(q, k, v, k_cache, v_cache, slots, pos, freq, qw, kw, q_out=out)
    want, keys = out.clone(), k_cache.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        lib.rope_append(q, k, v, k_cache, v_cache, slots, pos, freq, qw, kw, q_out=out)
    out.zero_()
    k_cache.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(k_cache.view(-1, 2, 128)[slots], keys.view(-1, 2, 128)[slots])
