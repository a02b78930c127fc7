"""The attention operators right behind kernels that write what they read, which they may start ahead of the end of: as if each had been
waited for."""
import pytest
import torch

from tests.test_gpu_tree_attention import Case as Attention
from tests.test_gpu_verify import Case as Verify

pytestmark = pytest.mark.gpu


def drafts():
    """A verification that takes long and whose results are contexts, positions and slots of what follows: sequence b's next token
    is 37 b, 1 or 2 drafts are kept."""
    c = Verify([3] * 24, 400000, "bf16", False, tree=False, temperature=[0.0])
    for b in range(24):
        c.logits[3 * b:3 * b + 3] = -1.0
        c.logits[3 * b, int(c.tokens[3 * b + 1])] = 5.0
        c.logits[3 * b + 1, int(c.tokens[3 * b + 2]) if b % 2 else 37 * b] = 5.0
        c.logits[3 * b + 2, 37 * b] = 9.0
    return c


@pytest.mark.parametrize("n,Hq", [(1, 4), (9, 8)])
def test_lengths_that_the_kernel_ahead_writes(lib, n, Hq):
    """The numbers of kept drafts as contexts."""
    v, c = drafts(), Attention([n] * 24, [5] * 24, Hq, 2, 64, 16, "bf16", False)
    outs = [torch.full((24,), 0, dtype=torch.int32, device="cuda"), torch.empty(24, 2, dtype=torch.int32, device="cuda"),
            torch.empty(24, dtype=torch.int64, device="cuda")]
    ws = lib.alloc_workspace(lib.tree_attention_workspace_bytes(24, n, Hq, 2, 64))
    got, want = torch.empty_like(c.q), torch.empty_like(c.q)

    def step(out, wait):
        outs[0].zero_()
        torch.cuda.synchronize()
        lib.verify_drafts(v.logits, v.tokens, v.parents, v.starts, v.u, v.uf, 3, temperature=v.heat, accepted=outs[0], path=outs[1], next_tokens=outs[2])
        if wait:
            torch.cuda.synchronize()
        lib.tree_attention(c.q, c.k, c.v, c.table, c.starts, outs[0], max_tokens=n, out=out, workspace=ws)
        torch.cuda.synchronize()
    step(want, True)
    assert outs[0].tolist() == [1, 2] * 12
    for _ in range(5):
        step(got, False)
        assert torch.equal(got, want)
    assert lib.get_last_error() == 0


@pytest.mark.parametrize("D", [64, 62])
def test_slots_and_positions_that_the_kernel_ahead_writes(lib, D):
    """The next tokens as positions and as slots."""
    v = drafts()
    g = torch.Generator(device="cuda").manual_seed(0)
    rows = torch.randn(24, 4, D, generator=g, device="cuda").bfloat16()
    freq = torch.logspace(0, -4, D // 2, device="cuda")
    following = torch.empty(24, dtype=torch.int64, device="cuda")

    def step(wait):
        caches = [torch.zeros(60, 16, 1, D, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        out = torch.empty(24, 2, D, dtype=torch.bfloat16, device="cuda")
        following.fill_(-1)
        torch.cuda.synchronize()
        lib.verify_drafts(v.logits, v.tokens, v.parents, v.starts, v.u, v.uf, 3, temperature=v.heat, next_tokens=following)
        if wait:
            torch.cuda.synchronize()
        lib.rope_append(rows[:, :2], rows[:, 2:3], rows[:, 3:], *caches, following, following, freq, q_out=out)
        torch.cuda.synchronize()
        return [out] + caches
    want = step(True)
    assert following.tolist() == [37 * b for b in range(24)] and want[1].any()
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(step(False), want))
    assert lib.get_last_error() == 0


def test_logits_that_the_kernel_ahead_writes(lib):
    """The head's product, then its verification."""
    g = torch.Generator(device="cuda").manual_seed(0)
    K, V = 4096, 32768
    codes = torch.randint(-2 ** 31, 2 ** 31 - 1, (V, K // 8), generator=g, device="cuda", dtype=torch.int64).int()
    blob = lib.prepack(codes, torch.full((K // 128, V), 0.02, dtype=torch.bfloat16, device="cuda"))
    v = Verify([3] * 5, V, "bf16", False)
    logits = torch.empty(15, V, dtype=torch.bfloat16, device="cuda")
    ws = lib.alloc_workspace(lib.workspace_bytes(15, V, K))

    def step(x, wait):
        logits.zero_()
        torch.cuda.synchronize()
        lib.mm(x, blob, V, out=logits, workspace=ws)
        if wait:
            torch.cuda.synchronize()
        return [t.clone() for t in lib.verify_drafts(logits, v.tokens, v.parents, v.starts, v.u, v.uf, 3)]
    for seed in range(5):
        x = torch.randn(15, K, generator=g, device="cuda").bfloat16()
        want = step(x, True)
        assert all(torch.equal(a, b) for a, b in zip(step(x, False), want))
    assert lib.get_last_error() == 0
