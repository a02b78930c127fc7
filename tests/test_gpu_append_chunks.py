"""Chunks of a prompt that give a thread several tokens one after the other, and warps some of whose lanes have no head.

Against the formulas in 64 bits on the GPU. Tolerance as in test_gpu_append."""
import pytest
import torch

from tests.test_gpu_append import TYPES, make

pytestmark = pytest.mark.gpu


def formula(x, weight, positions, freq, interleaved):
    """(features, the sizes of each pair) of [T][heads][D] in 64 bits."""
    x = x.double()
    if weight is not None:
        x = x / (x.square().mean(dim=2, keepdim=True) + 1e-6).sqrt() * weight.double()
    out, size = x.clone(), x.abs()
    if freq is not None:
        half = len(freq)
        a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
        w = positions.double()[:, None, None] * freq.double()
        p, q = x[..., a], x[..., b]
        out[..., a], out[..., b] = p * w.cos() - q * w.sin(), q * w.cos() + p * w.sin()
        size[..., a] = size[..., b] = p.abs() + q.abs()
    return out, size


@pytest.mark.parametrize("T,Hq,Hk,D,R,norm,interleaved,dtype", [
    (2500, 32, 8, 64, 64, True, False, "bf16"),      # one token's heads fill a CTA
    (2501, 32, 8, 128, 64, False, True, "fp16"),     # more heads than fit beside each other
    (20001, 2, 1, 32, 32, True, False, "bf16"),      # many tokens beside each other
    (60000, 1, 1, 64, 32, True, True, "fp16"),       # 12 lanes a token: 252 of a CTA's 256 have one
    (60001, 1, 1, 80, 0, True, False, "bf16"),
    (30011, 3, 1, 64, 64, True, False, "bf16"),
    (130000, 1, 1, 16, 16, True, False, "bf16"),     # one lane a head: 85 tokens beside each other
    (40003, 0, 3, 64, 64, True, False, "bf16"),      # keys and values alone
    (2, 1, 1, 16, 16, True, False, "bf16"),          # 6 lanes of 32
    (3, 1, 2, 48, 16, True, True, "fp16"),
])
def test_chunks(lib, T, Hq, Hk, D, R, norm, interleaved, dtype):
    rows, k_cache, v_cache, slots, pos, freq, (qw, kw) = make(T, Hq, Hk, D, R, dtype, norm, 16, seed=T)
    slots[T // 2] = -1                               # a padded token among the others
    q, k, v = (rows[:, :Hq] if Hq else None), rows[:, Hq:Hq + Hk], rows[:, Hq + Hk:]
    want_v = v_cache.view(-1, Hk, D).clone()
    before = k_cache.view(-1, Hk, D).clone()
    out = lib.rope_append(q, k, v, k_cache, v_cache, slots, pos, freq, q_weight=qw if Hq else None, k_weight=kw, eps=1e-6, interleaved=interleaved)
    assert lib.get_last_error() == 0
    eps, tiny = torch.finfo(TYPES[dtype]).eps, torch.finfo(TYPES[dtype]).tiny

    def near(got, want, size):
        off = (got.double() - want).abs() - (eps / 2 * want.abs() * (1 + eps) + 24 * 2.0 ** -24 * size + tiny * eps)
        assert off.max() <= 0, (off.max(), (off > 0).nonzero()[:4])
    if Hq:
        near(out, *formula(q, qw, pos, freq, interleaved))
    kept = slots >= 0
    near(k_cache.view(-1, Hk, D)[slots[kept]], *(x[kept] for x in formula(k, kw, pos, freq, interleaved)))
    want_v[slots[kept]] = v[kept]
    assert torch.equal(v_cache.view(-1, Hk, D), want_v)
    untouched = torch.ones(len(before), dtype=torch.bool, device="cuda")
    untouched[slots[kept]] = False
    assert torch.equal(k_cache.view(-1, Hk, D)[untouched], before[untouched])
