"""Verification of drafts against the fp64 oracle.

Decisions. A weight exp(x - max) errs by the roundings of x / temperature and the difference (2^-23 of up to 60 each, so 2 60 2^-23 =
2^-16 of the weight at most) and expf's 2 ulp; the oracle says how near a walk came to a border, and walks nearer than 1e-4 are
left out. The drawn token has to be one whose share of [0, 1) lies within 2^-15 of the random number; weights
err alike, and a running sum by no more than the weights in it do."""
import numpy as np
import pytest
import torch

from oracle import attention_oracle as A

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


class Case:
    def __init__(self, counts, V, dtype, probs, tree=True, seed=0, temperature=None, pad=0, spread=3.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.starts_list = np.concatenate([[0], np.cumsum(counts)]).astype(int)
        T = int(self.starts_list[-1])
        x = spread * torch.randn(T, V + pad, generator=g, device="cuda")
        self.logits = x.to(TYPES[dtype])[:, pad:]
        guess = torch.softmax(x[:, pad:] + torch.randn(T, V, generator=g, device="cuda"), dim=1) if T else x[:, pad:]
        self.q = guess if probs else None
        parents, tokens = [], []
        for b, n in enumerate(counts):
            s = self.starts_list[b]
            for i in range(n):
                p = -1 if i == 0 else int(rng.integers(max(0, i - 4), i)) if tree else i - 1
                parents.append(p)
                row = guess[s + max(p, 0)]
                top = row.topk(min(V, 4)).indices.tolist()
                tokens.append(int(torch.multinomial(row, 1, generator=g)) if probs else top[i % len(top)])
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")   # noqa: E731
        self.parents, self.starts = ints(parents), ints(self.starts_list)
        self.tokens = torch.tensor(tokens, dtype=torch.int64, device="cuda")
        self.u, self.uf = (torch.rand(k, generator=g, device="cuda") for k in (T, len(counts)))
        self.heat = None if temperature is None else torch.tensor([temperature[b % len(temperature)] for b in range(len(counts))], device="cuda")
        self.most = max(1, max(counts))

    def run(self, lib):
        out = lib.verify_drafts(self.logits, self.tokens, self.parents, self.starts, self.u, self.uf, self.most, draft_probs=self.q,
                                temperature=self.heat)
        assert lib.get_last_error() == 0
        return out

    def check(self, lib):
        accepted, path, after = (t.cpu().numpy() for t in self.run(lib))
        n = lambda t: None if t is None else t.cpu().numpy()   # noqa: E731
        logits, tokens, parents, u, uf, q, heat = self.logits.double().cpu().numpy(), n(self.tokens), n(self.parents), n(self.u), n(self.uf), n(self.q), n(self.heat)
        for b in range(len(self.starts_list) - 1):
            s = slice(self.starts_list[b], self.starts_list[b + 1])
            want, p, margin = A.verify(logits[s], tokens[s], parents[s], u[s], uf[b], None if q is None else q[s], 1.0 if heat is None else float(heat[b]))
            if margin <= 1e-4:
                continue
            assert path[b].tolist() == want + [-1] * (path.shape[1] - len(want)) and accepted[b] == len(want), b
            if p is None:
                assert after[b] == -1
                continue
            t = int(after[b])
            assert 0 <= t < len(p) and p[t] > 0
            upto = np.cumsum(p)
            lo, hi = (upto[t - 1] if t else 0.0), upto[t]
            assert lo - 2.0 ** -15 <= uf[b] <= hi + 2.0 ** -15, (b, t, lo, hi, uf[b])
        return accepted


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("probs", [False, True])
@pytest.mark.parametrize("V", [1, 2, 7, 33, 1000, 1025, 16384, 16385, 40001, 131072, 400000])
def test_vocabularies(lib, dtype, probs, V):
    if V == 1:                                       # (p of the only token is 1: uniforms below it keep every draft)
        Case([4, 1], V, dtype, probs).check(lib)
    else:
        Case([5, 1, 3], V, dtype, probs, seed=V % 1000, spread=1.5).check(lib)


@pytest.mark.parametrize("probs", [False, True])
@pytest.mark.parametrize("tree", [False, True])
def test_walks_of_many_kinds(lib, probs, tree):
    rng = np.random.default_rng(3)
    counts = rng.integers(0, 18, 300).tolist()
    accepted = Case(counts, 300, "fp32", probs, tree=tree, seed=4, temperature=[0.7, 0.0, 1.3, 1.0], spread=4.0).check(lib)
    assert accepted.max() >= 2 and (accepted == 0).any()


@pytest.mark.parametrize("pad", [1, 3, 8])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_rows_off_their_boundaries(lib, dtype, pad):
    Case([4, 2], 20000, dtype, True, pad=pad).check(lib)


def test_masked_logits(lib):
    """-inf and the type's lowest value; a draft that cannot occur; the last token alone possible."""
    c = Case([3, 3, 2, 2], 5000, "bf16", True, seed=2)
    x = c.logits
    x[0, 100:] = -float("inf")
    x[3] = torch.finfo(torch.bfloat16).min
    x[6] = -float("inf")
    x[6, 4999] = -3.0
    x[8, ::2] = -float("inf")
    c.check(lib)


def test_rows_without_a_distribution_end_the_walk(lib):
    c = Case([1, 1, 1, 2, 1], 3000, "fp32", False, seed=5, temperature=[1.0, 1.0, 1.0, 0.0, 0.0])
    c.logits[0] = -float("inf")
    c.logits[1, 17] = float("nan")
    c.logits[2, 2999] = float("inf")
    c.logits[3] = -1.0
    c.tokens[4], c.parents[4] = 0, 0                # the largest of equal logits is the first: the draft is kept
    c.logits[4, 5] = float("nan")
    accepted, path, after = c.run(lib)
    assert after.tolist()[:4] == [-1] * 4 and after[4] >= 0 and accepted.tolist() == [0, 0, 0, 1, 0]


def test_temperatures_that_cannot_be(lib):
    c = Case([2] * 6, 500, "fp32", False, temperature=[-1.0, float("nan"), float("inf"), 1e-40, 0.0, 1.0])
    accepted, path, after = c.run(lib)
    assert after.tolist()[:4] == [-1] * 4 and (after[4:] >= 0).all() and accepted.tolist()[:4] == [0] * 4


def test_greedy_ties_go_to_the_lowest_index(lib):
    for V in (40, 3000, 50000, 200000):
        c = Case([1, 1], V, "bf16", False, temperature=[0.0])
        c.logits.zero_()
        c.logits[1, V - 1] = 1.0
        c.logits[1, V // 2] = 1.0
        assert c.run(lib)[2].tolist() == [0, V // 2]


def test_borders_of_the_random_numbers(lib):
    """0 takes the first token with a weight, the largest float below 1 one of the last, and 1 itself the last one."""
    c = Case([1, 1, 1], 20001, "fp32", False, spread=0.0)
    c.logits[:, :3] = -float("inf")
    c.logits[:, 19999:] = -float("inf")
    c.uf.copy_(torch.tensor([0.0, 1 - 2.0 ** -24, 1.0]))
    assert c.run(lib)[2].tolist() == [3, 19998, 19998]
    even = Case([1], 4096, "fp32", False, spread=0.0)
    for k in (0, 1, 31, 32, 1023, 1024, 4095):
        even.uf.fill_(k / 4096)                      # exactly on a border: the token that begins there
        assert even.run(lib)[2].tolist() == [k]


def test_drafts_outside_the_vocabulary_and_odd_parents(lib):
    c = Case([6, 3], 100, "fp32", True, tree=False)
    before = c.run(lib)
    c.tokens[1] = -1
    c.tokens[7] = 100
    accepted, path, after = c.run(lib)
    assert accepted.tolist() == [0, 0] and (path == -1).all() and (after >= 0).all()
    c.parents[1:6] = torch.tensor([5, 7, -3, 4, 2 ** 31 - 1], dtype=torch.int32)
    assert c.run(lib)[0].tolist() == [0, 0]
    assert before[0].shape == accepted.shape


def test_a_draft_that_the_target_matches_is_kept(lib):
    """p = q keeps every draft (u < 1), and where p has the token's whole mass too."""
    c = Case([6, 4], 1000, "fp32", True, tree=False)
    c.q = torch.softmax(c.logits, dim=1)
    c.u.fill_(0.999)
    assert c.run(lib)[0].tolist() == [5, 3]
    c = Case([3], 1000, "fp32", False, tree=False)
    c.logits.fill_(-float("inf"))
    c.logits[torch.arange(2), c.tokens[1:]] = 0.0
    c.logits[2, 5] = 0.0
    assert c.run(lib)[0].tolist() == [2] and c.run(lib)[2].tolist() == [5]


def test_nothing_left_of_the_target(lib):
    """The draft's distribution covers the target's, its uniform says no: the target's own stands."""
    c = Case([2], 1000, "fp32", True, tree=False)
    c.q = 2 * torch.softmax(c.logits, dim=1)
    c.u.fill_(0.99)
    c.uf.fill_(0.5)
    accepted, path, after = c.run(lib)
    upto = torch.cumsum(torch.softmax(c.logits[0].double(), dim=0), dim=0)
    assert accepted.tolist() == [0] and abs(int(after) - int((upto > 0.5).int().argmax())) == 0


def test_starts_that_cannot_be_are_reported(lib):
    c = Case([2, 2], 100, "fp32", False)
    for starts in ([0, 2, 5], [-1, 2, 4], [0, 3, 4], [2, 0, 4], [2 ** 31 - 2, 2 ** 31 - 1, 2 ** 31 - 1]):
        c.starts.copy_(torch.tensor(starts, dtype=torch.int32))
        out = lib.verify_drafts(c.logits, c.tokens, c.parents, c.starts, c.u, c.uf, 2)
        assert lib.get_last_error() == lib.ERR_INVALID, starts
        assert (out[2] == -1).any()


def test_captured_and_the_same_every_time(lib):
    c = Case([5, 3, 9], 131072, "bf16", True, temperature=[0.8])
    want = [t.clone() for t in c.run(lib)]
    outs = [torch.zeros_like(t) for t in want]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        lib.verify_drafts(c.logits, c.tokens, c.parents, c.starts, c.u, c.uf, c.most, draft_probs=c.q, temperature=c.heat, accepted=outs[0],
                          path=outs[1], next_tokens=outs[2])
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
