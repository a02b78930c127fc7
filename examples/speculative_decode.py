"""Decodes with drafted trees on a small decoder made of this package's operators.

Each layer's projections are 4-bit (wq4.mm); between them lie wq4.rope_append (norms of queries and keys, rotation, the
paged cache) and wq4.tree_attention. Every step drafts a tree from the model without its layers (the
embedding through the head), runs the tree through the model in one pass, and wq4.verify_drafts says which drafts
stand and which token follows. Kept drafts that lie apart in the cache are moved together. Weights are random.

    python examples/speculative_decode.py [--batch 3] [--steps 8] [--features 256] [--layers 2] [--vocab 1024]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_only_quantized_wq4_gb300 as wq4  # noqa: E402

HEAD, PAGE = 64, 16
# the tree of each step: the last certain token, three guesses at the next one, and a chain behind the first of them
PARENTS = [-1, 0, 0, 0, 1, 4]


def tree(parents):
    """(masks, depths): a word for each token with the bits of those it descends from, and how many they are."""
    masks, depths = [], []
    for i, p in enumerate(parents):
        masks.append((masks[p] if p >= 0 else 0) | 1 << i)
        depths.append(depths[p] + 1 if p >= 0 else 0)
    return masks, depths


def weight4(n, k, g, scale=1.0):
    """A random weight of uint4b8 codes with a bf16 scale per 128 of k, prepacked."""
    codes = torch.randint(-2 ** 31, 2 ** 31 - 1, (n, k // 8), generator=g, device="cuda", dtype=torch.int64).int()
    scales = torch.full((k // 128, n), 0.2 * scale / k ** 0.5, dtype=torch.bfloat16, device="cuda")
    return wq4.prepack(codes, scales)


class Decoder:
    """The model and its paged caches, one table for all layers."""

    def __init__(self, features, layers, vocab, batch, places, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.features, self.vocab, self.batch = features, vocab, batch
        self.heads, self.kv_heads = features // HEAD, max(1, features // HEAD // 2)
        self.rows = (self.heads + 2 * self.kv_heads) * HEAD
        ones = lambda n: torch.ones(n, dtype=torch.bfloat16, device="cuda")   # noqa: E731
        self.embed = torch.randn(vocab, features, generator=g, device="cuda").bfloat16()
        self.layers = [dict(norm=ones(features), qkv=weight4(self.rows, features, g), q_norm=ones(HEAD), k_norm=ones(HEAD),
                            out=weight4(features, self.heads * HEAD, g)) for _ in range(layers)]
        self.norm, self.head = ones(features), weight4(vocab, features, g, scale=3.0)
        self.inv_freq = 1e4 ** (-torch.arange(0, HEAD, 2, device="cuda", dtype=torch.float32) / HEAD)
        width = -(-places // PAGE)
        self.table = torch.randperm(batch * width, generator=g, device="cuda").int().view(batch, width)
        self.caches = [[torch.zeros(batch * width, PAGE, self.kv_heads, HEAD, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
                       for _ in range(layers)]
        self.context = torch.zeros(batch, dtype=torch.int32, device="cuda")
        # for prompts and trees alike: calls on one stream share it, and the largest needs no less than the others
        self.workspace = wq4.alloc_workspace(wq4.tree_attention_workspace_bytes(batch, places, self.heads, self.kv_heads, HEAD))

    def slots(self, sequence, place):
        return self.table[sequence, place // PAGE].long() * PAGE + place % PAGE

    def logits(self, tokens, starts, sequence, place, position, max_tokens, mask=None):
        """Logits of tokens at their places of the sequences' caches."""
        h, y = self.embed[tokens], torch.empty(len(tokens), self.features, dtype=torch.bfloat16, device="cuda")
        slots, add = self.slots(sequence, place), None
        for layer, (k_cache, v_cache) in zip(self.layers, self.caches):
            _, _, summed = wq4.add_rmsnorm_quant(h, layer["norm"], residual=add, y=y)
            h = h if summed is None else summed
            rows = wq4.mm(y, layer["qkv"], self.rows).view(len(tokens), -1, HEAD)
            q, k, v = rows.split([self.heads, self.kv_heads, self.kv_heads], dim=1)
            q = wq4.rope_append(q, k, v, k_cache, v_cache, slots, position, self.inv_freq, layer["q_norm"], layer["k_norm"])
            o = wq4.tree_attention(q, k_cache, v_cache, self.table, starts, self.context, max_tokens=max_tokens, mask=mask,
                                   workspace=self.workspace)
            add = wq4.mm(o.view(len(tokens), -1), layer["out"], self.features)
        wq4.add_rmsnorm_quant(h, self.norm, residual=add, y=y)
        return wq4.mm(y, self.head, self.vocab)

    def prefill(self, prompts):
        """Runs prompts (a list of token lists) through the model; returns each one's last row of logits."""
        counts = [len(p) for p in prompts]
        tokens = torch.tensor([t for p in prompts for t in p], device="cuda")
        starts = torch.tensor([0] + counts, device="cuda").cumsum(0).int()
        sequence = torch.repeat_interleave(torch.arange(len(prompts), device="cuda"), torch.tensor(counts, device="cuda"))
        place = torch.arange(len(tokens), device="cuda") - starts[sequence]
        out = self.logits(tokens, starts, sequence, place, place, max(counts))
        self.context += torch.tensor(counts, dtype=torch.int32, device="cuda")
        return out[starts[1:].long() - 1]

    def draft(self, roots):
        """[batch][tree] tokens guessed by the model without layers."""
        y = torch.empty(len(roots), self.features, dtype=torch.bfloat16, device="cuda")

        def guess(tokens, k):
            wq4.add_rmsnorm_quant(self.embed[tokens], self.norm, y=y)
            return wq4.mm(y, self.head, self.vocab).topk(k, dim=1).indices
        first = guess(roots, 3)
        second = guess(first[:, 0], 1)
        third = guess(second[:, 0], 1)
        return torch.cat([roots[:, None], first, second, third], dim=1)

    def step(self, roots, temperature, g):
        """One drafted tree per sequence. Returns (tokens kept after each root, the next roots)."""
        B, n = len(roots), len(PARENTS)
        masks, depths = tree(PARENTS)
        each = lambda v, dtype: torch.tensor(v, dtype=dtype, device="cuda").repeat(B)   # noqa: E731
        drafts = self.draft(roots)
        tokens, parents = drafts.flatten(), each(PARENTS, torch.int32)
        starts = torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")
        sequence = torch.arange(B, device="cuda").repeat_interleave(n)
        context = self.context.long()[sequence]
        logits = self.logits(tokens, starts, sequence, context + each(range(n), torch.int64), context + each(depths, torch.int64), n,
                             each(masks, torch.int64)[:, None].contiguous())
        u = torch.rand(B * n + B, generator=g, device="cuda")
        accepted, path, following = wq4.verify_drafts(logits, tokens, parents, starts, u[:B * n], u[B * n:], n, temperature=temperature)
        # kept drafts are moved to the places behind the root; the reads are done before the writes
        kept = torch.arange(n - 1, device="cuda")[None] < accepted[:, None]
        who = torch.arange(B, device="cuda")[:, None].expand_as(path)[kept]
        start = self.context.long()[who]
        source, target = self.slots(who, start + path[kept]), self.slots(who, start + 1 + torch.arange(n - 1, device="cuda")[None].expand_as(path)[kept])
        for k_cache, v_cache in self.caches:
            for c in (k_cache, v_cache):
                flat = c.view(-1, self.kv_heads, HEAD)
                flat[target] = flat[source]
        self.context += 1 + accepted
        return [drafts[b, path[b, :int(accepted[b])].long()].tolist() for b in range(B)], following


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("batch", 3), ("steps", 8), ("features", 256), ("layers", 2), ("vocab", 1024)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    g = torch.Generator(device="cuda").manual_seed(1)
    prompts = [torch.randint(0, a.vocab, (5 + 3 * b,), generator=g, device="cuda").tolist() for b in range(a.batch)]
    model = Decoder(a.features, a.layers, a.vocab, a.batch, places=max(map(len, prompts)) + len(PARENTS) * (a.steps + 1))
    roots = model.prefill(prompts).argmax(dim=1)
    temperature = torch.tensor([0.0 if b % 2 == 0 else 0.8 for b in range(a.batch)], device="cuda")
    texts = [[int(r)] for r in roots]
    for _ in range(a.steps):
        kept, roots = model.step(roots, temperature, g)
        for text, more, root in zip(texts, kept, roots.tolist()):
            text += more + [root]
    assert wq4.get_last_error() == 0
    for b, text in enumerate(texts):
        print("sequence %d: %d tokens in %d steps:" % (b, len(text), a.steps), *text)


if __name__ == "__main__":
    main()
