"""Scores a sequence of tokens with a small decoder made of this package's operators alone.

Each layer keeps one projection at 4 bits and its feed-forward at 8: the norm before the 4-bit projection
writes 16-bit rows (wq4.mm), the one before the feed-forward writes 8-bit rows (wq4.block_mm), the gated
activation writes 8-bit rows for the second 8-bit product, and the head's logits go to
wq4.token_logprobs. Mixing along the sequence is a causal mean, which stands in for attention; weights are
random. Prints each token's log probability, the entropy and the likeliest alternatives.

    python examples/score_tokens.py [--tokens 32] [--features 512] [--layers 2] [--vocab 8000]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_only_quantized_wq4_gb300 as wq4  # noqa: E402

F8 = torch.float8_e4m3fn


def weight8(n, k, g):
    """A random weight as e4m3 codes [n][k] with a scale per 128 x 128 block."""
    nb, kb = -(-n // 128), -(-k // 128)
    w = torch.zeros(nb * 128, kb * 128, device="cuda")
    w[:n, :k] = torch.randn(n, k, generator=g, device="cuda") / k ** 0.5
    blocks = w.view(nb, 128, kb, 128)
    scales = (blocks.abs().amax(dim=(1, 3)) / 448).clamp_min(2.0 ** -126)
    codes = (blocks / scales[:, None, :, None]).view(nb * 128, kb * 128)[:n, :k]
    return codes.to(F8).contiguous(), scales.contiguous()


def weight4(n, k, g):
    """A random weight of uint4b8 codes with a bf16 scale per 128 of k, prepacked."""
    codes = torch.randint(-2 ** 31, 2 ** 31 - 1, (n, k // 8), generator=g, device="cuda", dtype=torch.int64).int()
    scales = torch.full((k // 128, n), 0.2 / k ** 0.5, dtype=torch.bfloat16, device="cuda")
    return wq4.prepack(codes, scales)


class Scorer:
    def __init__(self, features, hidden, layers, vocab, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        ones = lambda: torch.ones(features, dtype=torch.bfloat16, device="cuda")   # noqa: E731
        self.features, self.vocab = features, vocab
        self.embed = torch.randn(vocab, features, generator=g, device="cuda").bfloat16()
        self.layers = [dict(norm1=ones(), mix=weight4(features, features, g), norm2=ones(),
                            up=weight8(2 * hidden, features, g), down=weight8(features, hidden, g))
                       for _ in range(layers)]
        self.norm, self.head = ones(), weight8(vocab, features, g)

    def logits(self, tokens):
        h = self.embed[tokens]                             # the residual stream, bf16
        x = None                                           # what the last projection adds to it
        mean = torch.ones(len(tokens), len(tokens), device="cuda").tril()
        mean = (mean / mean.sum(dim=1, keepdim=True)).bfloat16()
        for layer in self.layers:
            y = torch.empty_like(h)
            if x is None:
                wq4.add_rmsnorm_quant(h, layer["norm1"], y=y)
            else:
                h = wq4.add_rmsnorm_quant(x, layer["norm1"], residual=h, y=y)[2]
            x = wq4.mm((mean @ y).contiguous(), layer["mix"], self.features)
            q, s, h = wq4.add_rmsnorm_quant(x, layer["norm2"], residual=h)
            q, s = wq4.silu_mul_quant(wq4.block_mm(q, s, *layer["up"]))
            x = wq4.block_mm(q, s, *layer["down"])
        q, s, _ = wq4.add_rmsnorm_quant(x, self.norm, residual=h)
        return wq4.block_mm(q, s, *self.head, dtype=torch.float32)

    def score(self, tokens, top_k=5):
        """(log probability of each next token, entropy, top ids, top log probabilities)"""
        return wq4.token_logprobs(self.logits(tokens)[:-1], tokens[1:].contiguous(), top_k=top_k)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=32)
    ap.add_argument("--features", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=1280)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--vocab", type=int, default=8000)
    a = ap.parse_args()
    wq4.build()
    model = Scorer(a.features, a.hidden, a.layers, a.vocab)
    tokens = torch.randint(0, a.vocab, (a.tokens,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    lp, ent, ids, tlp = model.score(tokens)
    if wq4.get_last_error():
        raise SystemExit("a kernel reported an error")
    for i, t in enumerate(tokens[1:].tolist()):
        best = ", ".join("%d %.2f" % z for z in zip(ids[i].tolist(), tlp[i].tolist()))
        print("token %6d  log p %7.3f  entropy %6.3f  likeliest: %s" % (t, float(lp[i]), float(ent[i]), best))
    print("log probability of the sequence: %.3f" % float(lp.sum()))


if __name__ == "__main__":
    main()
