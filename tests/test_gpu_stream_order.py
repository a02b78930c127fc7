"""Buffers that are written and read again by calls close behind one another, as a decode loop reuses them, in programmatic
dependent launches: every call reads what the one ahead of it wrote, and nothing older."""
import pytest
import torch

from tests.test_gpu_block_mm import operand, scale_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 20, 70, 300])
def test_reused_buffers(lib, T):
    """norm -> product -> log probabilities over one set of buffers, with other inputs each time, against the same calls
    with a synchronisation between any two."""
    D, V, n = 640, 3000, 12
    g = torch.Generator(device="cuda").manual_seed(T)
    xs = [(torch.randn(T, D, generator=g, device="cuda") * 4.0 ** (i % 3)).bfloat16() for i in range(n)]
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    ws = [(torch.rand(D, generator=g, device="cuda") + 0.5 + i).bfloat16() for i in range(n)]
    _, head = operand(V, D, 2)
    _, hs = scale_rows(-(-V // 128), 5, 3, 5)
    tokens = torch.randint(0, V, (T,), generator=g, device="cuda")
    q, s = lib.alloc_quant_rows(T, D)
    logits = torch.empty(T, V, device="cuda")

    def loop(sync):
        out = []
        for i in range(n):
            lib.add_rmsnorm_quant(xs[i], ws[i], q=q, scales=s)
            sync()
            lib.block_mm(q, s, head, hs, out=logits)
            sync()
            out.append(lib.token_logprobs(logits, tokens, top_k=4))
            sync()
            lib.block_mm(q, s, head, hs, out=logits)
            sync()
            out.append(lib.token_logprobs(logits, tokens, top_k=4))
            sync()
        torch.cuda.synchronize()
        assert lib.get_last_error() == 0
        return out

    want = loop(torch.cuda.synchronize)
    for _ in range(5):
        for a, b in zip(loop(lambda: None), want):
            assert all(torch.equal(p, r) for p, r in zip(a, b))
    assert not torch.equal(want[0][0], want[2][0])


def test_float_zero_sums_of_reused_rows(lib):
    """The 4-bit product with float zeros reads rows that the norm ahead of it wrote into the same buffer again and again."""
    M, N, K, n = 80, 256, 512, 10
    g = torch.Generator(device="cuda").manual_seed(5)
    codes = torch.randint(-2 ** 31, 2 ** 31 - 1, (N, K // 8), generator=g, device="cuda", dtype=torch.int64).int()
    scales = (torch.rand(K // 128, N, generator=g, device="cuda") * 0.02).bfloat16()
    zeros = torch.randn(K // 128, N, generator=g, device="cuda").bfloat16()
    blob = lib.prepack(codes, scales, zeros, qtype="u4_fzp")
    xs = [torch.randn(M, K, generator=g, device="cuda").bfloat16() for _ in range(n)]
    ws = [(torch.rand(K, generator=g, device="cuda") + i).bfloat16() for i in range(n)]
    y = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    q, s = lib.alloc_quant_rows(M, K)
    work = lib.alloc_workspace(lib.workspace_bytes(M, N, K, qtype="u4_fzp"))

    def loop(sync):
        out = []
        for i in range(n):
            lib.add_rmsnorm_quant(xs[i], ws[i], q=q, scales=s, y=y)
            sync()
            out.append(lib.mm(y, blob, N, qtype="u4_fzp", workspace=work))
            sync()
        torch.cuda.synchronize()
        assert lib.get_last_error() == 0
        return out

    want = loop(torch.cuda.synchronize)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(loop(lambda: None), want))
