"""Attention of drafted tokens over a paged cache against the fp64 oracle.

Tolerance, with eps the type's and per row spread = sum p |v|, size = max scale sum |q k|. Probabilities are rounded to the
type ahead of the product with the values (eps / 2 of spread) and the result once more (eps / 2 of it). A score is a sum of D
exact products added up in groups of 16 by the tensor cores, each addition off by at most 2^-22 of the sum of sizes (they
cut where fp32 would round): (D / 16 + 2) 2^-22 size, twice where a probability is measured against the sum; exp2 adds 2^-21.
Sums over the places are fp32 in groups of 16 as well, and joined: (L / 16 + 64) 2^-22 of spread at most."""
import numpy as np
import pytest
import torch

from oracle import attention_oracle as A

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def tree(n, seed):
    """bool [n][n]: which tokens each of a random tree's sees."""
    rng = np.random.default_rng(seed)
    seen = np.zeros((n, n), dtype=bool)
    for i in range(n):
        if i:
            seen[i] = seen[rng.integers(max(0, i - 5), i)]
        seen[i, i] = True
    return seen


def words(mask, T, n):
    """int64 [T][ceil(n / 64)] of a list of bool rows."""
    out = np.zeros((T, -(-n // 64)), dtype=np.uint64)
    for t, row in enumerate(mask):
        for j in np.flatnonzero(row):
            out[t, j // 64] |= np.uint64(1) << np.uint64(j % 64)
    return torch.from_numpy(out.view(np.int64)).cuda()


class Case:
    def __init__(self, counts, context, Hq, Hk, D, page, dtype, masked, seed=0, extra_rows=0, slack=2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        dt = TYPES[dtype]
        self.dtype, self.counts, self.context_list, self.D = dtype, counts, context, D
        self.starts_list = np.concatenate([[0], np.cumsum(counts)]).astype(int)
        T = int(self.starts_list[-1]) + extra_rows
        need = [-(-(c + n) // page) for c, n in zip(context, counts)]
        pages = sum(need) + slack
        order = torch.randperm(pages, generator=g, device="cuda").tolist()
        width = max(max(need), 1) + 1
        table, at = [], 0
        for k in need:
            table.append(order[at:at + k] + [-7] * (width - k))            # (entries past a sequence's places are not read)
            at += k
        self.k, self.v = (torch.randn(pages, page, Hk, D, generator=g, device="cuda").to(dt) for _ in "kv")
        self.q = (1.5 * torch.randn(T, Hq, D, generator=g, device="cuda")).to(dt)
        self.table = torch.tensor(table, dtype=torch.int32, device="cuda")
        self.starts = torch.tensor(self.starts_list, dtype=torch.int32, device="cuda")
        self.context = torch.tensor(context, dtype=torch.int32, device="cuda")
        self.most = max(max(counts), 1)
        self.seen = [row for b, n in enumerate(counts) for row in tree(n, seed + b)] if masked else None
        self.mask = words(self.seen, T, self.most) if masked else None

    def stale(self, value):
        """Puts a value into every place that is no sequence's."""
        used = torch.zeros(self.k.shape[:2], dtype=torch.bool, device="cuda")
        page = self.k.shape[1]
        for b, (c, n) in enumerate(zip(self.context_list, self.counts)):
            p = torch.arange(c + n, device="cuda")
            used[self.table[b].long()[p // page], p % page] = True
        self.k[~used], self.v[~used] = value, value

    def oracle(self, scale=None):
        n = lambda t: t.cpu().numpy()   # noqa: E731
        return A.tree_attention(self.q.double().cpu().numpy(), self.k.double().cpu().numpy(), self.v.double().cpu().numpy(), n(self.table),
                                self.starts_list, self.context_list, self.seen, self.D ** -0.5 if scale is None else scale)

    def run(self, lib, lse=True, **kw):
        T, H, _ = self.q.shape
        out = torch.full_like(self.q, 7.0, memory_format=torch.contiguous_format)
        lse = torch.full((T, H), 7.0, device="cuda") if lse else None
        lib.tree_attention(self.q, self.k, self.v, self.table, self.starts, self.context, max_tokens=self.most, mask=self.mask, out=out,
                           lse=lse, **kw)
        assert lib.get_last_error() == 0
        return out, lse

    def check(self, lib, scale=None, **kw):
        out, lse = self.run(lib, scale=scale, **kw)
        want, want_lse, spread, size = self.oracle(scale)
        self.compare(out, lse, want, want_lse, spread, size)
        return out, lse

    def compare(self, out, lse, want, want_lse, spread, size):
        n = int(self.starts_list[-1])
        got, eps, L = out.double().cpu().numpy(), torch.finfo(TYPES[self.dtype]).eps, max(c + k for c, k in zip(self.context_list, self.counts))
        arg = (self.D / 16 + 2) * 2.0 ** -22 * size + 2.0 ** -21
        tol = eps / 2 * (np.abs(want) + spread) * (1 + eps) + spread * (2 * arg[..., None] + (L / 16 + 64) * 2.0 ** -22) + 2.0 ** -25
        with np.errstate(invalid="ignore"):
            off = ~((np.abs(got - want) <= tol) | (got == want) | (np.isnan(got) & np.isnan(want)))[:n]
        assert not off.any(), (np.argwhere(off)[:5], got[:n][off][:5], want[:n][off][:5])
        l_got = lse.double().cpu().numpy()
        with np.errstate(invalid="ignore"):
            l_tol = arg + (L / 16 + 64) * 2.0 ** -22 + 2.0 ** -22 * np.abs(want_lse)
            l_off = ~((np.abs(l_got - want_lse) <= l_tol) | (l_got == want_lse) | (np.isnan(l_got) & np.isnan(want_lse)))[:n]
        assert not l_off.any(), (np.argwhere(l_off)[:5], l_got[:n][l_off][:5], want_lse[:n][l_off][:5])
        # rows that are no sequence's are left as they were
        assert (got[n:] == 7).all() and (l_got[n:] == 7).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("context", [0, 1, 15, 16, 63, 64, 65, 200, 700])
def test_single_tokens(lib, dtype, context):
    Case([1], [context], 8, 2, 64, 16, dtype, False, seed=context).check(lib)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("D", [8, 40, 64, 80, 96, 128, 136, 192, 200, 256])
def test_head_sizes(lib, dtype, D):
    Case([3, 1], [130, 70], 4, 2, D, 32, dtype, True, seed=D).check(lib)


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (2, 2), (7, 1), (14, 2), (16, 1), (17, 1), (12, 3), (40, 1)])
@pytest.mark.parametrize("n", [1, 5])
def test_head_groups(lib, Hq, Hk, n):
    Case([n, n, max(1, n - 2)], [33, 300, 0], Hq, Hk, 64, 48, "bf16", n > 1, seed=Hq).check(lib)


@pytest.mark.parametrize("page", [16, 32, 48, 64, 80, 128, 256])
@pytest.mark.parametrize("masked", [False, True])
def test_page_sizes(lib, page, masked):
    Case([4, 6], [page - 2, 3 * page + 1], 4, 2, 128, page, "bf16", masked, seed=page).check(lib)


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("n", [2, 16, 31, 63, 64, 65, 130])
def test_trees_and_chains(lib, masked, n):
    Case([n, 1, max(1, n // 2)], [90, 5, 0], 8, 2, 64, 16, "bf16", masked, seed=n).check(lib)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("D", [64, 128])
def test_long_and_ragged(lib, dtype, D):
    """Lengths that several CTAs share, beside short ones; empty sequences between."""
    counts, context = [1, 0, 3, 2, 0, 1, 7, 1], [9000, 400, 12, 2500, 0, 0, 1111, 64]
    Case(counts, context, 8, 2, D, 16, dtype, True, seed=1, extra_rows=3).check(lib)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("counts,context,Hq,Hk", [([32, 1], [40000, 3000], 4, 1), ([50], [30000], 8, 1), ([16, 3], [300, 20000], 4, 2)])
def test_trees_over_long_contexts(lib, dtype, D, counts, context, Hq, Hk):
    """So many tiles for each CTA that every buffer is used many times over; every sixth token is compared."""
    c = Case(counts, context, Hq, Hk, D, 64, dtype, True, seed=2)
    out, lse = c.run(lib)
    keep = range(0, sum(counts), 6)
    q, K, V, page = c.q, c.k.double().cpu().numpy(), c.v.double().cpu().numpy(), 64
    parts = [np.zeros(x, dtype=np.float64) for x in (q.shape, q.shape[:2], q.shape, q.shape[:2])]
    for t in keep:
        b = int(np.searchsorted(c.starts_list, t, side="right")) - 1
        places = np.concatenate([np.arange(context[b]), context[b] + np.flatnonzero(c.seen[t])])
        pages = c.table[b].cpu().numpy()[places // page]
        x = q[t].double().cpu().numpy()
        for h in range(Hq):
            k, v = K[pages, places % page, h * Hk // Hq], V[pages, places % page, h * Hk // Hq]
            s = D ** -0.5 * (k @ x[h])
            p = np.exp(s - s.max())
            parts[1][t, h] = s.max() + np.log(p.sum())
            p /= p.sum()
            parts[0][t, h], parts[2][t, h] = p @ v, p @ np.abs(v)
            parts[3][t, h] = D ** -0.5 * (np.abs(k) @ np.abs(x[h])).max()
    drop = np.setdiff1d(np.arange(sum(counts)), list(keep))
    out, lse = out.clone(), lse.clone()
    for t in drop:                                   # (not compared)
        out[t], lse[t] = 0, 0
    c.compare(out, lse, *parts)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("D", [8, 40, 64, 72, 80, 96, 128])
@pytest.mark.parametrize("counts,context", [([12, 3, 40], [130, 0, 300]), ([5, 6, 0, 4, 5, 1], [33, 700, 9, 127, 128, 129])])
def test_many_rows_of_head_sizes(lib, dtype, D, counts, context):
    """More rows than one tile of 16 takes, of a whole batch: tiles of 128 rows, filled twice, once and in part."""
    Case(counts, context, 16, 2, D, 16, dtype, True, seed=D, extra_rows=2).check(lib)


@pytest.mark.parametrize("page", [16, 48, 64, 80, 128, 256])
@pytest.mark.parametrize("masked", [False, True])
def test_many_rows_of_page_sizes(lib, page, masked):
    Case([9, 20, 7], [page - 2, 3 * page + 1, 2 * page], 8, 2, 128, page, "bf16", masked, seed=page).check(lib)


@pytest.mark.parametrize("group", [3, 7, 12, 64, 129])
def test_many_rows_of_groups(lib, group):
    """Rows of one token in two tiles, and tokens that end inside one."""
    Case([11, 2, 6, 1, 9], [60, 190, 0, 500, 128], group * 2, 2, 64, 32, "bf16", True, seed=group).check(lib)


@pytest.mark.parametrize("scale", [0.0, -0.2, 2.5, 40.0])
def test_many_rows_scales(lib, scale):
    Case([11, 20, 6], [60, 190, 0], 8, 2, 64, 32, "bf16", True).check(lib, scale=scale)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), 3e38])
def test_many_rows_stale_places(lib, value):
    c = Case([30, 41, 3], [130, 7, 500], 16, 2, 64, 16, "bf16", True, slack=3)
    want = c.run(lib)
    c.stale(value)
    got = c.run(lib)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", list(TYPES))
def test_many_rows_values_that_are_not_finite(lib, dtype):
    """Drafted values, keys and the context's, in tiles that one CTA takes and that several share."""
    c = Case([30, 41, 9], [140, 3000, 0], 16, 2, 128, 16, dtype, True, seed=7)

    def at(b, place):
        return c.table[b, place // 16].long(), place % 16
    c.v[(*at(0, 140 + 2), 0, 3)] = float("inf")
    c.v[(*at(0, 140 + 3), 1, 100)] = float("nan")
    c.v[(*at(1, 3000 + 7), 0, 127)] = -float("inf")
    c.k[(*at(1, 3000 + 9), 1, 5)] = float("nan")
    c.v[(*at(1, 17), 1, 64)] = float("nan")
    out, lse = c.check(lib)
    assert not torch.isfinite(out).all() and torch.isfinite(out).any()


def test_many_rows_that_see_nothing(lib):
    c = Case([40, 30], [0, 20], 8, 2, 64, 16, "bf16", True)
    for t in (1, 39, 45):
        c.seen[t] = np.zeros(len(c.seen[t]), dtype=bool)
    c.mask = words(c.seen, 70, 40)
    out, lse = c.check(lib)
    assert (out[1] == 0).all() and torch.isneginf(lse[39]).all()


def test_many_sequences(lib):
    rng = np.random.default_rng(0)
    counts, context = rng.integers(0, 4, 400).tolist(), rng.integers(0, 90, 400).tolist()
    Case(counts, context, 2, 1, 64, 16, "bf16", False).check(lib)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), 3e38])
@pytest.mark.parametrize("n,Hq,context", [(1, 4, 100), (5, 4, 60), (40, 8, 333)])
def test_stale_places_do_not_count(lib, value, n, Hq, context):
    c = Case([n, max(1, n - 1)], [context, 7], Hq, 2, 64, 16, "bf16", n > 1, slack=3)
    want = c.run(lib)
    c.stale(value)
    got = c.run(lib)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n,Hq,D", [(6, 4, 64), (20, 8, 128)])
def test_masked_values_that_are_not_finite(lib, dtype, n, Hq, D):
    """A drafted token's NaN or infinity reaches the tokens that see it, and no other."""
    c = Case([n], [40], Hq, 2, D, 16, dtype, True, seed=5)
    place = lambda i: (c.table[0, (40 + i) // 16].long(), (40 + i) % 16)   # noqa: E731
    page, at = place(2)
    c.v[page, at, 0, 3] = float("inf")
    c.v[page, at, 1, 5] = -float("inf")
    page, at = place(3)
    c.v[page, at, 0, 4] = float("nan")
    page, at = place(4)
    c.k[page, at, 1, 7] = float("nan")
    out, lse = c.check(lib)
    assert not torch.isfinite(out).all() and torch.isfinite(out).any()


def test_values_of_the_context_that_are_not_finite(lib):
    c = Case([3], [70], 4, 2, 64, 16, "bf16", True, seed=6)
    c.v[c.table[0, 1].long(), 3, 0, 9] = float("nan")
    c.check(lib)


@pytest.mark.parametrize("n,Hq", [(5, 4), (40, 8)])
def test_rows_that_see_nothing(lib, n, Hq):
    """Masks that name nothing, without a context: zeros and -inf. Bits past the tokens count for nothing."""
    c = Case([n, n], [0, 20], Hq, 2, 64, 16, "bf16", True)
    c.seen[1] = np.zeros(n, dtype=bool)
    c.seen[n - 1] = np.zeros(n, dtype=bool)
    c.seen[n + 2] = np.zeros(n, dtype=bool)
    c.mask = words(c.seen, 2 * n, n)
    c.mask[1] |= torch.tensor(-(1 << 62), device="cuda")
    out, lse = c.check(lib)
    assert (out[1] == 0).all() and torch.isneginf(lse[1]).all() and (out[n - 1] == 0).all()


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.7, 30.0])
def test_scales(lib, scale):
    Case([4], [150], 4, 2, 64, 16, "bf16", True).check(lib, scale=scale)


def test_strided_tensors(lib):
    """Heads ahead of tokens in q and out, heads ahead of places in the cache, keys and values in one tensor."""
    c = Case([5, 2], [77, 130], 8, 4, 64, 16, "bf16", True)
    want, want_lse = c.run(lib)
    both = torch.stack([c.k, c.v], dim=1).permute(0, 1, 3, 2, 4).contiguous()      # [pages][2][heads][places][D]
    c.k, c.v = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
    c.q = c.q.transpose(0, 1).contiguous().transpose(0, 1)
    wide = torch.zeros(8, c.q.shape[0], 72, dtype=torch.bfloat16, device="cuda")
    out = wide[:, :, :64].transpose(0, 1)
    lib.tree_attention(c.q, c.k, c.v, c.table, c.starts, c.context, max_tokens=c.most, mask=c.mask, out=out)
    assert torch.equal(out, want) and (wide[:, :, 64:] == 0).all()


@pytest.mark.parametrize("counts", [[1, 1, 1], [1, 9, 2], [30, 9, 64]])
def test_the_same_bits_every_time_and_the_workspace_lasts(lib, counts):
    c = Case(counts, [5000, 800, 90], 16, 2, 128, 16, "bf16", len(set(counts)) > 1)
    ws = lib.alloc_workspace(lib.tree_attention_workspace_bytes(3, c.most, 16, 2, 128))
    first = c.run(lib, workspace=ws)
    for _ in range(5):
        again = c.run(lib, workspace=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_captured_with_lengths_that_change(lib):
    """A captured call reads lengths, tables and masks when it is replayed."""
    c = Case([2, 3], [700, 90], 8, 2, 128, 16, "bf16", True, slack=80)
    ws = lib.alloc_workspace(lib.tree_attention_workspace_bytes(2, c.most, 8, 2, 128))
    table = torch.arange(2 * 60, dtype=torch.int32, device="cuda").view(2, 60) % c.k.shape[0]
    out = torch.empty_like(c.q)

    def call():
        lib.tree_attention(c.q, c.k, c.v, table, c.starts, c.context, max_tokens=c.most, mask=c.mask, out=out, workspace=ws)
    call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for lengths in ([700, 90], [3, 900], [0, 0], [64, 65]):
        c.context.copy_(torch.tensor(lengths, dtype=torch.int32))
        out.zero_()
        graph.replay()
        got = out.clone()
        call()
        assert torch.equal(got, out), lengths
    assert lib.get_last_error() == 0


@pytest.mark.parametrize("n,Hq", [(2, 4), (40, 16)])
def test_pages_and_lengths_that_cannot_be_are_reported(lib, n, Hq):
    c = Case([n, n], [50, 20], Hq, 2, 64, 16, "bf16", False)
    args = (c.q, c.k, c.v)
    good = lib.tree_attention(*args, c.table, c.starts, c.context, max_tokens=n)
    assert lib.get_last_error() == 0
    for page in (-1, c.k.shape[0], c.k.shape[0] + 1, 2 ** 31 - 1, -2 ** 31):
        table = c.table.clone()
        table[0, 1] = page
        lib.tree_attention(*args, table, c.starts, c.context, max_tokens=n)
        assert lib.get_last_error() == lib.ERR_INVALID, page
    for context in ([50, -1], [c.table.shape[1] * 16 - n + 1, 20], [2 ** 31 - 1, 20], [2 ** 30, 20], [-2 ** 31, 20]):
        lib.tree_attention(*args, c.table, c.starts, torch.tensor(context, dtype=torch.int32, device="cuda"), max_tokens=n)
        assert lib.get_last_error() == lib.ERR_INVALID, context
    for starts in ([0, n, 2 * n + 1], [-1, n, 2 * n], [0, n + 1, 2 * n], [0, 2 * n, n], [2 ** 31 - 2, 2 ** 31 - 1, 2 ** 31 - 1],
                   [-2 ** 31, 2 ** 31 - 1, 2 * n]):
        lib.tree_attention(*args, c.table, torch.tensor(starts, dtype=torch.int32, device="cuda"), c.context, max_tokens=n)
        assert lib.get_last_error() == lib.ERR_INVALID, starts
    assert torch.equal(good, lib.tree_attention(*args, c.table, c.starts, c.context, max_tokens=n))
    assert lib.get_last_error() == 0


def test_a_workspace_too_small_is_refused(lib):
    c = Case([1], [50], 4, 2, 64, 16, "bf16", False)
    n = lib.tree_attention_workspace_bytes(1, 1, 4, 2, 64)
    with pytest.raises(lib.Wq4Error) as e:
        lib.tree_attention(c.q, c.k, c.v, c.table, c.starts, c.context, workspace=lib.alloc_workspace(n)[:n - 16])
    assert e.value.status == lib.ERR_WORKSPACE


@pytest.mark.parametrize("counts", [[1, 2], [40, 30]])
def test_a_wait_that_runs_out_is_reported(lib, counts):
    """One wait per CTA that nothing ends: the call stops early, and the next one is as ever."""
    c = Case(counts, [900, 90], 8, 2, 64, 16, "bf16", False)
    want = c.run(lib)
    lib.set_option(lib.OPT_TEST_STALL, 1)
    lib.set_option(lib.OPT_TIMEOUT_CYCLES, 2000000)
    try:
        lib.tree_attention(c.q, c.k, c.v, c.table, c.starts, c.context, max_tokens=c.most)
        assert lib.get_last_error() == lib.ERR_TIMEOUT
    finally:
        lib.set_option(lib.OPT_TEST_STALL, 0)
        lib.set_option(lib.OPT_TIMEOUT_CYCLES, 0)
    got = c.run(lib)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
