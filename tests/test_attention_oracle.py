"""The attention operators' fp64 oracle against torch on the CPU, and the walk's distribution. Runs without a GPU."""
import numpy as np
import torch

from oracle import attention_oracle as A


def test_rotation_turns_pairs_and_keeps_lengths():
    rng = np.random.default_rng(0)
    x, f = rng.standard_normal(16), 1e4 ** (-np.arange(4) / 4)
    for interleaved in (False, True):
        y = A.rotate(x, 7, f, interleaved)
        assert np.allclose(y[8:], x[8:])
        pairs = [(2 * i, 2 * i + 1) if interleaved else (i, i + 4) for i in range(4)]
        for (a, b), w in zip(pairs, 7 * f):
            z = complex(x[a], x[b]) * np.exp(1j * w)
            assert np.allclose([y[a], y[b]], [z.real, z.imag])


def test_attention_matches_torch_on_a_chain():
    rng = np.random.default_rng(1)
    B, H, G, D, page = 2, 4, 2, 8, 16
    counts, context = [3, 2], [20, 0]
    starts = np.array([0, 3, 5])
    table = np.array([[3, 1], [0, 2]])
    K, V = rng.standard_normal((2, 4, page, H // G, D))
    q = rng.standard_normal((5, H, D))
    out, lse, spread, size = A.tree_attention(q, K, V, table, starts, context, None, 0.3)
    for b in range(B):
        n, c = counts[b], context[b]
        k = K[table[b]].reshape(-1, H // G, D)[:c + n].repeat(G, axis=1)
        v = V[table[b]].reshape(-1, H // G, D)[:c + n].repeat(G, axis=1)
        hide = torch.ones(n, c + n, dtype=torch.bool).triu(c + 1)
        s = torch.einsum("thd,phd->htp", torch.from_numpy(q[starts[b]:starts[b + 1]]), torch.from_numpy(k)) * 0.3
        s = s.masked_fill(hide, -torch.inf)
        want = torch.einsum("htp,phd->thd", s.softmax(-1), torch.from_numpy(v))
        assert np.allclose(out[starts[b]:starts[b + 1]], want.numpy())
        assert np.allclose(lse[starts[b]:starts[b + 1]], s.logsumexp(-1).t().numpy())
    mask = np.zeros((5, 3), dtype=bool)
    out, lse, _, _ = A.tree_attention(q, K, V, table, starts, [0, 0], mask, 0.3)
    assert not out.any() and np.isneginf(lse).all()


def test_a_walks_tokens_are_distributed_as_the_targets():
    """The first token that follows the root, kept draft or drawn, over many random numbers."""
    rng = np.random.default_rng(2)
    V, runs = 5, 20000
    logits = rng.standard_normal((3, V)) * 1.5
    target = np.exp(logits[0] / 0.8) / np.exp(logits[0] / 0.8).sum()
    q = rng.dirichlet(np.ones(V), size=3)
    seen = np.zeros((2, V))
    for _ in range(runs):
        for with_q in (0, 1):
            drafts = rng.choice(V, 2, p=q[0]) if with_q else rng.choice(V, 2, replace=False)
            tokens = [0, *drafts]                  # two children of the root
            path, p, _ = A.verify(logits, tokens, [-1, 0, 0], rng.random(3), 0.0, q if with_q else None, 0.8)
            first = tokens[path[0]] if path else int(np.searchsorted(np.cumsum(p), rng.random() * p.sum(), side="right"))
            seen[with_q, min(first, V - 1)] += 1
    # five standard deviations of a share
    assert (np.abs(seen / runs - target) < 5 * np.sqrt(target / runs)).all(), (seen / runs, target)


def test_greedy_walks_follow_the_largest():
    logits = np.array([[0, 3, 3, 1.0], [5, 0, 0, 0], [0, 0, 0, 9]])
    path, p, _ = A.verify(logits, [0, 2, 1], [-1, 0, 0], [0.9, 0.9, 0.9], 0.5, None, 0.0)
    assert path == [2] and np.argmax(p) == 3
    assert A.verify(np.full((1, 4), -np.inf), [0], [-1], [0.0], 0.0)[1] is None
