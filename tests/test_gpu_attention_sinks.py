"""One place takes nearly all of a row's probability and its value is zero: what the other places add is the whole output.

Their probabilities are far below the largest, and are rounded to the type ahead of the product with the values. fp16 has 2^-14 as its
least normal number and steps of 2^-24 below it, so they are held times a power of two: the largest of a row as 2^13 or more. A
probability is then off by half a step, 2^-11 of it, or by 2^-25 / 2^13 = 2^-38 of the row's largest, whichever is more. bf16
has fp32's range."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_tree_attention import TYPES, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n,Hq,D", [(1, 4, 64), (3, 4, 192), (40, 8, 64), (40, 8, 128)])
@pytest.mark.parametrize("nats", [6.0, 12.0, 17.5, 18.5])
@pytest.mark.parametrize("last", [False, True])
def test_places_far_below_the_largest(lib, dtype, n, Hq, D, nats, last):
    """The large score comes first of all (the reference stays) or behind the others (what they added is scaled down)."""
    context = 40000
    c = Case([n], [context], Hq, 2, D, 64, dtype, False, seed=n + D)
    c.q = 0.05 * c.q
    c.q[..., 0] = 8.0
    c.k[..., 0] = 0.0
    c.v = (c.v.float() + 1.0).to(TYPES[dtype])
    place = context - 1 if last else 0
    at = c.table[0, place // 64].long(), place % 64
    c.k[at] = 0.0
    c.k[(*at, slice(None), 0)] = nats * math.sqrt(D) / 8
    c.v[at] = 0.0
    out, lse = c.run(lib)
    got, f = out.double().cpu().numpy(), lambda t: t.double().cpu().numpy()   # noqa: E731
    pages = c.table[0].long()[torch.arange(context + n, device="cuda") // 64]
    K, V = (f(t[pages, torch.arange(context + n, device="cuda") % 64]) for t in (c.k, c.v))
    q, eps = f(c.q), torch.finfo(TYPES[dtype]).eps
    for t in range(0, n, 7):
        for h in range(Hq):
            k, v = K[:context + t + 1, h // (Hq // 2)], V[:context + t + 1, h // (Hq // 2)]
            s = k @ q[t, h] * D ** -0.5
            p = np.exp(s - s.max())
            z = p.sum()
            want, spread = p @ v / z, p @ np.abs(v) / z
            # the roundings of scores and sums as in test_gpu_tree_attention; p's, and the result's, half steps
            size = D ** -0.5 * (np.abs(k) @ np.abs(q[t, h])).max()
            arg = (D / 16 + 2) * 2.0 ** -22 * size + 2.0 ** -21
            low = 2.0 ** -38 * np.abs(v).sum(0) / z if dtype == "fp16" else 0.0
            out_step = np.maximum(eps / 2 * np.abs(want), 2.0 ** -25 if dtype == "fp16" else 0.0)
            tol = out_step + eps / 2 * spread * (1 + eps) + low + spread * (2 * arg + (context / 16 + 64) * 2.0 ** -22)
            assert (np.abs(got[t, h] - want) <= tol).all(), (t, h, np.abs(got[t, h] - want).max(), want[:3], got[t, h, :3])
            assert abs(float(lse[t, h]) - (s.max() + math.log(z))) <= arg + (context / 16 + 64) * 2.0 ** -22 + 2.0 ** -22 * abs(s.max() + math.log(z))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n,Hq", [(2, 4), (40, 8)])
@pytest.mark.parametrize("scale", [0.125, 1.0, 9.0])
def test_rows_whose_maximum_grows_on_the_way(lib, dtype, n, Hq, scale):
    """Scores that rise along the context, a little and much at a time, over all that several CTAs share."""
    context = 6000
    c = Case([n], [context], Hq, 2, 64, 64, dtype, n > 2, seed=3)
    rise = torch.linspace(-2, 2, context, device="cuda")
    places = torch.arange(context, device="cuda")
    c.q[..., 1] = 2.0
    c.k[c.table[0].long()[places // 64], places % 64, :, 1] = rise[:, None].to(c.k.dtype)
    c.check(lib, scale=scale)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n,Hq", [(1, 4), (40, 16)])
def test_one_place_with_all_the_weight(lib, dtype, n, Hq):
    """Its probability is 1, which every type holds: what comes out is its value to the bit, as all else lies 100 nats below."""
    context = 500
    c = Case([n, n], [context, context], Hq, 2, 64, 16, dtype, False, seed=n)
    c.q[..., 0] = 8.0
    c.k[..., 0] = 0.0
    for b in range(2):
        c.k[c.table[b, 3].long(), 5, :, 0] = 113.0 + 0.37 * b
    out, lse = c.run(lib)
    for b in range(2):
        want = c.v[c.table[b, 3].long(), 5].repeat_interleave(Hq // 2, dim=0)
        assert torch.equal(out[b * n:(b + 1) * n], want.expand(n, Hq, 64))
