"""The attention kernel for many rows per kv head where test_gpu_tree_attention's cases go to the other one; each call is seen to
take the kernel it is meant for."""
import numpy as np
import pytest
import torch

from tests.test_gpu_tree_attention import TYPES, Case, words

pytestmark = pytest.mark.gpu


@pytest.fixture
def by_tiles(lib, capfd):
    """Runs a call and holds it to units of 256 rows."""
    def call(f, rows=256):
        capfd.readouterr()
        lib.set_option(lib.OPT_TRACE, 1)
        try:
            r = f()
        finally:
            lib.set_option(lib.OPT_TRACE, 0)
        said = [x for x in capfd.readouterr().err.splitlines() if "tree_attention" in x]
        assert said and all(x.split()[-1] == "rows=%d" % rows for x in said), said
        return r
    return call


@pytest.mark.parametrize("page", [16, 48, 64, 80, 96, 128, 256])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_page_sizes(lib, by_tiles, page, masked, D):
    c = Case([9, 20, 7, 1, 12, 3], [page - 2, 3 * page + 1, 2 * page, 0, 700, 127], 8, 2, D, page, "bf16", masked, seed=page)
    by_tiles(lambda: c.check(lib))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("scale", [0.01, 1.0, 2.5, 40.0])
def test_scales(lib, by_tiles, dtype, scale):
    c = Case([11, 20, 6, 9, 17, 5], [60, 190, 0, 900, 128, 3000], 8, 2, 64, 32, dtype, True)
    by_tiles(lambda: c.check(lib, scale=scale))


@pytest.mark.parametrize("scale", [0.0, -0.2])
def test_scales_that_the_other_kernel_takes(lib, by_tiles, scale):
    c = Case([11, 20, 6, 9, 17, 5], [60, 190, 0, 900, 128, 3000], 8, 2, 64, 32, "bf16", True)
    by_tiles(lambda: c.check(lib, scale=scale), rows=16)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("group", [1, 3, 5])
def test_small_groups(lib, by_tiles, dtype, group):
    c = Case([23, 40, 6, 31, 9], [60, 190, 0, 500, 128], group * 4, 4, 64, 32, dtype, True, seed=group)
    by_tiles(lambda: c.check(lib))


def test_more_sequences_than_threads(lib, by_tiles):
    """Their lengths are summed up in rounds; empty sequences at the start, the end and in between."""
    rng = np.random.default_rng(0)
    counts, context = rng.integers(0, 4, 1500), rng.integers(0, 60, 1500)
    counts[:40], counts[700:760], counts[-30:] = 0, 0, 0
    c = Case(counts.tolist(), context.tolist(), 8, 1, 64, 16, "bf16", False, extra_rows=5)
    by_tiles(lambda: c.check(lib))


def test_long_context_of_few_units(lib, by_tiles):
    """A wide table sends few units here."""
    c = Case([5], [20000], 8, 2, 64, 64, "bf16", True)
    by_tiles(lambda: c.check(lib))


def test_a_long_chain(lib, by_tiles):
    """A prompt: every token sees those before it."""
    c = Case([2000, 300], [0, 170], 4, 1, 64, 64, "bf16", False)
    by_tiles(lambda: c.check(lib))


def test_words_of_masks(lib, by_tiles):
    """Masks of several words, places that begin anywhere in a tile."""
    c = Case([200, 129, 64, 65], [1, 63, 127, 128], 4, 2, 64, 16, "bf16", True)
    by_tiles(lambda: c.check(lib))


def test_captured_with_lengths_that_change(lib, by_tiles):
    c = Case([20, 33, 6], [700, 90, 0], 8, 2, 128, 16, "bf16", True, slack=300)
    ws = lib.alloc_workspace(lib.tree_attention_workspace_bytes(3, c.most, 8, 2, 128))
    c.table = torch.arange(3 * 200, dtype=torch.int32, device="cuda").view(3, 200) % c.k.shape[0]
    out = torch.empty_like(c.q)

    def call():
        lib.tree_attention(c.q, c.k, c.v, c.table, c.starts, c.context, max_tokens=c.most, mask=c.mask, out=out, workspace=ws)
    by_tiles(call)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for lengths in ([700, 90, 0], [3, 2900, 65], [0, 0, 0], [128, 129, 127]):
        c.context.copy_(torch.tensor(lengths, dtype=torch.int32))
        c.context_list = lengths
        out.zero_()
        graph.replay()
        got = out.clone()
        call()
        assert torch.equal(got, out), lengths
        want, want_lse, spread, size = c.oracle()
        lse = torch.from_numpy(want_lse).float()
        c.compare(got, lse, want, want_lse, spread, size)
    assert lib.get_last_error() == 0


@pytest.mark.parametrize("D", [136, 192, 256])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_large_heads_of_many_rows(lib, by_tiles, D, dtype):
    """Heads above 128: more than one unit of 16 rows, more tiles than the ring has slots, parts of several CTAs."""
    c = Case([40, 9, 1], [700, 2500, 0], 8, 2, D, 48, dtype, True, seed=D)
    by_tiles(lambda: c.check(lib), rows=16)


@pytest.mark.parametrize("D", [192, 256])
def test_large_heads_over_a_long_context(lib, by_tiles, D):
    c = Case([2], [30000], 2, 1, D, 64, "bf16", True, seed=D)
    by_tiles(lambda: c.check(lib), rows=16)
