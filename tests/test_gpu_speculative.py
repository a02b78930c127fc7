"""The attention operators run one after the other, as a decode step with drafts runs them: the example, and a chain of steps each
of which is held against the fp64 oracle on what the kernels before it left."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import attention_oracle as A

pytestmark = pytest.mark.gpu
HALF_STEP = torch.finfo(torch.bfloat16).eps / 2
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import speculative_decode
    finally:
        sys.path.pop(0)
    return speculative_decode


def test_example_prints_a_line_per_sequence(lib):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "speculative_decode.py"), "--steps", "4"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.count("tokens in 4 steps") == 3


def test_caches_after_steps_are_those_of_the_whole_text(lib):
    """Steps with kept and dropped drafts, then one more token's logits: those of the whole text run through at once. The two go
    through other kernels (tiles, splits of sums) and round every layer's rows to bf16 there, steps of 2^-8 that two
    layers and a head carry on: 0.05 of the logits' norm is five times what a few such steps add up to."""
    E = example()
    g = torch.Generator(device="cuda").manual_seed(4)
    prompts = [torch.randint(0, 512, (n,), generator=g, device="cuda").tolist() for n in (3, 17, 30)]
    model = E.Decoder(256, 2, 512, 3, places=120, seed=2)
    roots = model.prefill(prompts).argmax(dim=1)
    texts = [list(p) for p in prompts]
    heat = torch.tensor([0.0, 1.0, 2.0], device="cuda")
    total = 0
    for _ in range(6):
        old = roots.tolist()
        kept, roots = model.step(roots, heat, g)
        total += sum(map(len, kept))
        for text, root, more in zip(texts, old, kept):
            text += [root] + more
    assert total > 0 and model.context.tolist() == [len(t) for t in texts]
    B = torch.arange(3, device="cuda")
    place = model.context.long()
    one = model.logits(roots, torch.arange(4, dtype=torch.int32, device="cuda"), B, place, place, 1)
    whole = E.Decoder(256, 2, 512, 3, places=120, seed=2).prefill([t + [r] for t, r in zip(texts, roots.tolist())])
    assert lib.get_last_error() == 0
    off = (one.float() - whole.float()).norm(dim=1) / whole.float().norm(dim=1)
    assert (off < 0.05).all(), off


@pytest.mark.parametrize("heads,kv_heads,D", [(8, 2, 64), (4, 4, 128)])
def test_a_step_against_the_oracle(lib, heads, kv_heads, D):
    """A prompt and a drafted tree through projection, append, attention, projection and verification."""
    sp = example()
    PARENTS = sp.PARENTS
    g = torch.Generator(device="cuda").manual_seed(3)
    E, V, page, context, n = 256, 384, 16, 37, len(PARENTS)
    rows = (heads + 2 * kv_heads) * D
    w_in, w_out = sp.weight4(rows, E, g), sp.weight4(V, heads * D, g, scale=6.0)
    k_cache, v_cache = (torch.zeros(8, page, kv_heads, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    table = torch.randperm(8, generator=g, device="cuda").int().view(2, 4)
    freq = 1e4 ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float32) / D)
    weight = torch.ones(D, dtype=torch.bfloat16, device="cuda")

    def project(x, sequence, place, position):
        y = lib.mm(x, w_in, rows).view(len(x), -1, D)
        q, k, v = y.split([heads, kv_heads, kv_heads], dim=1)
        slots = table[sequence, place // page].long() * page + place % page
        before = k_cache.double().cpu().numpy(), v_cache.double().cpu().numpy()
        q_out = lib.rope_append(q, k, v, k_cache, v_cache, slots, position, freq, weight, weight)
        f = lambda t: t.double().cpu().numpy()   # noqa: E731
        want = A.rope_append(f(q), f(k), f(v), *before, slots.cpu().numpy(), position.cpu().numpy(), f(freq), f(weight), f(weight), 1e-6, False)
        for got, ref in zip((q_out, k_cache, v_cache), want):
            # Half a step of the value: bf16 holds 7 bits behind the first, neighbours lie 2^-7 of the power of two below them apart, and
            # a rounding is off by at most half of that, 2^-8 of the value. And fp32's roundings of a head's features, at
            # most sqrt(D) in size behind the norm.
            assert (np.abs(f(got) - ref) <= HALF_STEP * np.abs(ref) * (1 + HALF_STEP) + 24 * 2.0 ** -24 * 2 * D ** 0.5).all()
        return q_out
    # the prompts' keys and values, then the trees
    both = torch.arange(2, device="cuda")
    sequence, place = both.repeat_interleave(context), torch.arange(context, device="cuda").repeat(2)
    project(torch.randn(2 * context, E, generator=g, device="cuda").bfloat16(), sequence, place, place)
    sequence = both.repeat_interleave(n)
    bits, depth = sp.tree(PARENTS)
    mask = [[bool(m >> j & 1) for j in range(n)] for m in bits]
    place = context + torch.arange(n, device="cuda").repeat(2)
    q = project(torch.randn(2 * n, E, generator=g, device="cuda").bfloat16(), sequence, place,
                context + torch.tensor(depth, device="cuda").repeat(2))
    starts, ctx = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda"), torch.full((2,), context, dtype=torch.int32, device="cuda")
    words = torch.tensor(bits, device="cuda").repeat(2)[:, None].contiguous()
    out = lib.tree_attention(q, k_cache, v_cache, table, starts, ctx, max_tokens=n, mask=words)
    want, _, spread, size = A.tree_attention(q.double().cpu().numpy(), k_cache.double().cpu().numpy(), v_cache.double().cpu().numpy(),
                                             table.cpu().numpy(), [0, n, 2 * n], [context, context], mask * 2, D ** -0.5)
    tol = HALF_STEP * 1.01 * (np.abs(want) + spread) + spread * (2 * (D / 16 + 2) * 2.0 ** -22 * size[..., None] + 2.0 ** -15)
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()
    # the head's logits decide on the drafts
    logits = lib.mm(out.view(2 * n, -1), w_out, V)
    tokens = torch.randint(0, V, (2 * n,), generator=g, device="cuda")
    tokens[1], tokens[n + 2] = logits[0].argmax(), logits[n].argmax()
    parents = torch.tensor(PARENTS, dtype=torch.int32, device="cuda").repeat(2)
    u, last = torch.rand(2 * n, generator=g, device="cuda"), torch.rand(2, generator=g, device="cuda")
    accepted, path, following = lib.verify_drafts(logits, tokens, parents, starts, u, last, n)
    assert lib.get_last_error() == 0
    for b in range(2):
        s = slice(b * n, (b + 1) * n)
        kept, p, margin = A.verify(logits[s].double().cpu().numpy(), tokens[s].tolist(), PARENTS, u[s].tolist(), float(last[b]))
        assert margin > 1e-4 and path[b].tolist()[:len(kept)] == kept and int(accepted[b]) == len(kept)
        upto = np.cumsum(p)
        t = int(following[b])
        assert (upto[t - 1] if t else 0) - 2.0 ** -15 <= float(last[b]) <= upto[t] + 2.0 ** -15

