"""The attention operators at the ends of what their arguments may be: offsets past 32 bits, a cache that is one page, batches of nothing,
rows ahead of the first sequence."""
import pytest
import torch

from tests.test_gpu_tree_attention import Case
from tests.test_gpu_verify import Case as Verify

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,Hq", [(1, 8), (40, 8)])
def test_caches_past_32_bits(lib, n, Hq):
    """Pages more than 2^32 elements from the first, against the same pages in a small cache; keys and values are put there by rope_append."""
    page, Hk, D = 64, 4, 128
    c = Case([n, n], [300, 17000], Hq, Hk, D, page, "bf16", n > 1)
    pages = 2 ** 32 // (page * Hk * D) + len(c.k) + 1
    far = pages - len(c.k)
    k, v = (torch.empty(pages, page, Hk, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    k[far:], v[far:] = c.k, c.v
    table = torch.where(c.table >= 0, c.table + far, c.table)
    rows = torch.randn(5, Hk, D, device="cuda").bfloat16()
    slots = torch.tensor([0, 1, 70, 127, 64 * len(c.k) - 1], device="cuda")

    def step(kc, vc, table, slots):
        lib.rope_append(None, rows, rows, kc, vc, slots)
        out, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:2], device="cuda")
        lib.tree_attention(c.q, kc, vc, table, c.starts, c.context, max_tokens=n, mask=c.mask, out=out, lse=lse)
        return out, lse
    got = step(k, v, table, slots + far * page)
    again = step(c.k, c.v, c.table, slots)
    assert lib.get_last_error() == 0
    assert torch.equal(k[far:], c.k) and torch.equal(v[far:], c.v)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_logits_past_32_bits(lib):
    """A sequence whose rows lie more than 2^32 elements from the first; the sequences ahead of it are empty."""
    V = 400000
    c = Verify([4], V, "bf16", True, seed=3)
    T = 2 ** 32 // V + 10
    x, q = torch.empty(T, V, dtype=torch.bfloat16, device="cuda"), torch.empty(T, V, device="cuda")
    x[-4:], q[-4:] = c.logits, c.q
    z = lambda t: torch.cat([torch.zeros(T - 4, dtype=t.dtype, device="cuda"), t])   # noqa: E731
    starts = torch.tensor([T - 4, T - 4, T - 4, T], dtype=torch.int32, device="cuda")
    want = c.run(lib)
    got = lib.verify_drafts(x, z(c.tokens), z(c.parents), starts, z(c.u), torch.cat([c.uf, c.uf, c.uf]), 4, draft_probs=q)
    assert lib.get_last_error() == 0
    assert got[0][2] == want[0][0] and torch.equal(got[1][2], want[1][0]) and got[2][2] == want[2][0]
    assert got[0][:2].tolist() == [0, 0] and got[2][:2].tolist() == [-1, -1] and (got[1][:2] == -1).all()


@pytest.mark.parametrize("n,Hq", [(1, 4), (3, 4), (60, 16)])
def test_a_page_for_a_whole_sequence(lib, n, Hq):
    """A cache without paging: [batch][places][heads][D], a table of one column."""
    c = Case([n, n, n], [900, 0, 1500], Hq, 2, 64, 2048, "bf16", n > 1)
    c.table = c.table[:, :1].contiguous()
    c.check(lib)


@pytest.mark.parametrize("n,Hq", [(1, 4), (40, 16)])
def test_nothing_but_empty_sequences(lib, n, Hq):
    c = Case([n, n], [100, 5], Hq, 2, 64, 16, "bf16", False)
    for at in (0, 2 * n):
        c.starts.fill_(at)
        out, lse = c.run(lib)
        assert (out == 7).all() and (lse == 7).all()


@pytest.mark.parametrize("n,Hq", [(2, 4), (40, 16)])
def test_rows_ahead_of_the_first_sequence(lib, n, Hq):
    c = Case([n, n, n], [100, 5, 70], Hq, 2, 64, 16, "bf16", True)
    want, want_lse = c.run(lib)
    out, lse = torch.full_like(want, 7.0), torch.full_like(want_lse, 7.0)
    lib.tree_attention(c.q, c.k, c.v, c.table[1:], c.starts[1:].clone(), c.context[1:].clone(), max_tokens=n, mask=c.mask, out=out, lse=lse)
    assert lib.get_last_error() == 0
    assert (out[:n] == 7).all() and (lse[:n] == 7).all() and torch.equal(out[n:], want[n:]) and torch.equal(lse[n:], want_lse[n:])


def test_verification_of_nothing(lib):
    z = lambda *s, dtype=torch.int32: torch.zeros(*s, dtype=dtype, device="cuda")   # noqa: E731
    for B in (0, 3):
        out = lib.verify_drafts(z(0, 1000, dtype=torch.bfloat16), z(0, dtype=torch.int64), z(0), z(B + 1), z(0, dtype=torch.float32),
                                z(B, dtype=torch.float32), 4)
        assert lib.get_last_error() == 0
        assert out[0].tolist() == [0] * B and (out[1] == -1).all() and out[2].tolist() == [-1] * B


def test_two_streams_at_once(lib):
    """Calls that overlap, a workspace each."""
    cases = [Case([n, 5], [9000, 700], 8, 2, 128, 16, "bf16", True, seed=n) for n in (40, 1)]
    want = [c.run(lib) for c in cases]
    spaces = [lib.alloc_workspace(lib.tree_attention_workspace_bytes(2, c.most, 8, 2, 128)) for c in cases]
    outs = [torch.empty_like(c.q) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s, ws, out in zip(cases, streams, spaces, outs):
            with torch.cuda.stream(s):
                lib.tree_attention(c.q, c.k, c.v, c.table, c.starts, c.context, max_tokens=c.most, mask=c.mask, out=out, workspace=ws)
    torch.cuda.synchronize()
    assert lib.get_last_error() == 0
    assert all(torch.equal(a, b[0]) for a, b in zip(outs, want))
