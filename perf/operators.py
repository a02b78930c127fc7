"""The 8-bit operators beside the W4A16 product, each as one measured pass.

  norm      h = x + residual; y = h / sqrt(mean(h^2) + eps) * weight, in e4m3 with a scale for each token
            and 128 features (what the product below reads), and h itself for the next layer
  gated     y = silu(gate) * up, in e4m3 with the same scales
  product   Y = X . W^T of e4m3 operands, X with a scale for each token and 128 of K, W with one for each
            block of 128 x 128
  logprobs  log probabilities of given tokens, the entropy of each row and its most likely tokens

`run` computes them with elementary torch operations in 32 bits or, with `own`, through the package.
Scales are laid out [blocks of 128][tokens], as the package's products read them.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126
BLOCK = 128
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one token of one sequence being decoded, ahead of the first projection of a layer
        {"name": "norm_1x4096_bf16", "op": "norm", "tokens": 1, "features": 4096, "residual": True, "dtype": "bf16"},
        # a ragged batch of short prompts at a width that ends inside a block of 128; the first layer
        # (nothing to add yet)
        {"name": "norm_517x2064_fp16", "op": "norm", "tokens": 517, "features": 2064, "residual": False, "dtype": "fp16"},
        # a chunk of a long prompt
        {"name": "norm_4096x4096_bf16", "op": "norm", "tokens": 4096, "features": 4096, "residual": True, "dtype": "bf16"},
        # a decode batch between the two projections of a feed-forward layer
        {"name": "gated_16x14336_bf16", "op": "gated", "tokens": 16, "features": 14336, "dtype": "bf16"},
        # the same layer for a chunk of a prompt
        {"name": "gated_4096x14336_bf16", "op": "gated", "tokens": 4096, "features": 14336, "dtype": "bf16"},
        # one token's projection: the weights are read once and used once
        {"name": "product_1x4096x4096_bf16", "op": "product", "M": 1, "N": 4096, "K": 4096, "dtype": "bf16"},
        # a decode batch through a feed-forward projection
        {"name": "product_16x14336x4096_bf16", "op": "product", "M": 16, "N": 14336, "K": 4096, "dtype": "bf16"},
        # a few short prompts, an output width that no tile divides and a K that ends inside a block
        {"name": "product_333x4100x2064_fp16", "op": "product", "M": 333, "N": 4100, "K": 2064, "dtype": "fp16"},
        # a chunk of a long prompt through the second feed-forward projection
        {"name": "product_4096x4096x14336_bf16", "op": "product", "M": 4096, "N": 4096, "K": 14336, "dtype": "bf16"},
        # one sampled token with its alternatives, from a head that answers in 32 bits
        {"name": "logprobs_1x131072_fp32", "op": "logprobs", "tokens": 1, "vocab": 131072, "top": 20, "masked": False, "dtype": "fp32"},
        # a decode batch under a grammar: most of the vocabulary is ruled out
        {"name": "logprobs_257x32001_fp16", "op": "logprobs", "tokens": 257, "vocab": 32001, "top": 5, "masked": True, "dtype": "fp16"},
        # scoring a prompt
        {"name": "logprobs_2048x131072_bf16", "op": "logprobs", "tokens": 2048, "vocab": 131072, "top": 20, "masked": False, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "gated", "product", "product", "logprobs"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "norm" or op == "gated":
        features = _log_int(rng, 64, 16384 if op == "norm" else 14336)
        if rng.random() < 0.5:                               # as often a whole number of blocks as not
            features = -(-features // BLOCK) * BLOCK
        tokens = _log_int(rng, 1, min(8192, 4096 * (4096 if op == "norm" else 14336) // features))
        case = {"op": op, "tokens": tokens, "features": features, "dtype": dtype}
        if op == "norm":
            case["residual"] = rng.random() < 0.75
        return case
    if op == "product":
        N, K = _log_int(rng, 64, 16384), _log_int(rng, 8, 1024) * 16
        if rng.random() < 0.5:
            N, K = -(-N // BLOCK) * BLOCK, -(-K // BLOCK) * BLOCK
        M = _log_int(rng, 1, max(1, min(4096, 4096 * 4096 * 14336 // (N * K))))
        return {"op": op, "M": M, "N": N, "K": K, "dtype": rng.choice(["bf16", "fp16", "fp32"])}
    vocab = _log_int(rng, 1000, 160000)
    tokens = _log_int(rng, 1, min(2048, 2048 * 131072 // vocab))
    return {"op": op, "tokens": tokens, "vocab": vocab, "top": rng.randint(1, 32), "masked": rng.random() < 0.3,
            "dtype": rng.choice(["bf16", "fp16", "fp32"])}


def _blocks(n):
    return -(-n // BLOCK)


def _pad(n, m):
    return -(-n // m) * m


def _quantised_rows(y):
    """(e4m3 [T][D], scales [ceil(D/128)][T]) of y [T][D] in 32 bits."""
    T, D = y.shape
    nb = _blocks(D)
    yb = torch.nn.functional.pad(y, (0, nb * BLOCK - D)).view(T, nb, BLOCK)
    scales = (yb.abs().amax(dim=2) / E4M3_MAX).clamp_min(SCALE_MIN)
    q = (yb / scales.unsqueeze(2)).view(T, nb * BLOCK)[:, :D]
    return q.to(torch.float8_e4m3fn), scales.t()


def _row_buffers(T, D):
    """Buffers for quantised rows as the products read them: rows padded to 16 bytes, scale rows to 4 tokens."""
    q = torch.empty((T, _pad(D, 16)), dtype=torch.float8_e4m3fn, device="cuda")[:, :D]
    s = torch.empty((_blocks(D), _pad(T, 4)), dtype=torch.float32, device="cuda")[:, :T]
    return q, s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    st = {"case": case}
    if op == "norm":
        T, D = case["tokens"], case["features"]
        # a few features of the hidden state are much larger than the others
        spread = torch.exp(0.5 * normal(D)) * torch.where(torch.rand(D, generator=g, device="cuda") < 0.005, 20.0, 1.0)
        st["x"] = normal(T, D).to(dt)
        st["residual"] = (normal(T, D) * spread).to(dt) if case["residual"] else None
        st["weight"] = (1.0 + 0.2 * normal(D)).to(dt)
        st["eps"] = 1e-5
        st["q"], st["scales"] = _row_buffers(T, D)
        st["h"] = torch.empty((T, D), dtype=dt, device="cuda") if case["residual"] else None
    elif op == "gated":
        T, D = case["tokens"], case["features"]
        st["x"] = (normal(T, 2 * D) * 1.5).to(dt)
        st["q"], st["scales"] = _row_buffers(T, D)
    elif op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        st["x"], st["x_scales"] = _row_buffers(M, K)
        q, s = _quantised_rows(normal(M, K) * torch.exp(0.5 * normal(K)))
        st["x"].copy_(q)
        st["x_scales"].copy_(s)
        nb, kb = _blocks(N), _blocks(K)
        w = torch.zeros((nb * BLOCK, kb * BLOCK), device="cuda")
        w[:N, :K] = normal(N, K) * (torch.exp(0.3 * normal(N, 1)) / math.sqrt(K))
        wb = w.view(nb, BLOCK, kb, BLOCK)
        ws = (wb.abs().amax(dim=(1, 3)) / E4M3_MAX).clamp_min(SCALE_MIN)
        wq = (wb / ws[:, None, :, None]).view(nb * BLOCK, kb * BLOCK)[:N, :K]
        st["w"], st["w_scales"] = wq.to(torch.float8_e4m3fn).contiguous(), ws.contiguous()
        st["y"] = torch.empty((M, N), dtype=dt, device="cuda")
    else:
        T, V, k = case["tokens"], case["vocab"], case["top"]
        # a hidden state's logits: a broad body and some tens of tokens that the context favours
        x = normal(T, V) * 2.0
        at = torch.randint(0, V, (T, 40), generator=g, device="cuda")
        x.scatter_add_(1, at, 8.0 + 3.0 * normal(T, 40))
        favoured = at[:, 0].clone()
        if case["masked"]:
            keep = torch.rand(T, V, generator=g, device="cuda") < 0.1
            keep.scatter_(1, favoured[:, None], True)
            x = torch.where(keep, x, torch.full_like(x, -math.inf))
        st["logits"] = x.to(dt)
        other = torch.randint(0, V, (T,), generator=g, device="cuda")
        likely = torch.rand(T, generator=g, device="cuda") < 0.8
        st["tokens"] = torch.where(likely, favoured, other)
        st["logprobs"] = torch.empty(T, dtype=torch.float32, device="cuda")
        st["entropy"] = torch.empty(T, dtype=torch.float32, device="cuda")
        st["top_ids"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
        st["top_logprobs"] = torch.empty((T, k), dtype=torch.float32, device="cuda")
    return st


def _run_own(st):
    import weight_only_quantized_wq4_gb300 as wq4
    op = st["case"]["op"]
    if op == "norm":
        wq4.add_rmsnorm_quant(st["x"], st["weight"], residual=st["residual"], eps=st["eps"], q=st["q"],
                              scales=st["scales"], residual_out=st["h"])
        out = {"q": st["q"], "scales": st["scales"]}
        if st["h"] is not None:
            out["h"] = st["h"]
        return out
    if op == "gated":
        wq4.silu_mul_quant(st["x"], q=st["q"], scales=st["scales"])
        return {"q": st["q"], "scales": st["scales"]}
    if op == "product":
        return wq4.block_mm(st["x"], st["x_scales"], st["w"], st["w_scales"], out=st["y"])
    wq4.token_logprobs(st["logits"], st["tokens"], top_k=st["case"]["top"], logprobs=st["logprobs"],
                       entropy=st["entropy"], top_ids=st["top_ids"], top_logprobs=st["top_logprobs"])
    return {"logprobs": st["logprobs"], "entropy": st["entropy"], "top_ids": st["top_ids"],
            "top_logprobs": st["top_logprobs"]}


def _ranked(x, k):
    """Indices of each row's k largest values, the lowest index first among equal ones."""
    b = x.view(torch.int32).to(torch.int64)
    b = torch.where(b < 0, -(1 << 31) - b, b)                # whole numbers in the order of the floats
    at = torch.arange(x.shape[1], device=x.device, dtype=torch.int64)
    key = (b << 32) + ((1 << 32) - 1 - at)
    best = torch.topk(key, k, dim=1).values
    return (1 << 32) - 1 - (best & ((1 << 32) - 1))


def run(st):
    if own:
        return _run_own(st)
    op, dt = st["case"]["op"], DTYPES[st["case"]["dtype"]]
    if op == "norm":
        h = st["x"].float()
        if st["residual"] is not None:
            h = h + st["residual"].float()
        y = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + st["eps"]) * st["weight"].float()
        q, s = _quantised_rows(y)
        out = {"q": q, "scales": s}
        if st["residual"] is not None:
            out["h"] = h.to(dt)
        return out
    if op == "gated":
        D = st["case"]["features"]
        gate, up = st["x"][:, :D].float(), st["x"][:, D:].float()
        q, s = _quantised_rows(gate / (1.0 + torch.exp(-gate)) * up)
        return {"q": q, "scales": s}
    if op == "product":
        N, K = st["w"].shape
        x = st["x"].float() * st["x_scales"].t().repeat_interleave(BLOCK, dim=1)[:, :K]
        w = st["w"].float() * st["w_scales"].repeat_interleave(BLOCK, dim=0)[:N].repeat_interleave(BLOCK, dim=1)[:, :K]
        return (x @ w.t()).to(dt)
    x = st["logits"].float()
    top = x.amax(dim=1, keepdim=True)
    e = torch.exp(x - top)
    z = e.sum(dim=1, keepdim=True)
    logp = x - top - torch.log(z)
    lp = logp.gather(1, st["tokens"][:, None])[:, 0]
    p = e / z
    entropy = -torch.where(p > 0, p * logp, torch.zeros_like(p)).sum(dim=1)
    ids = _ranked(x, st["case"]["top"])
    return {"logprobs": lp, "entropy": entropy, "top_ids": ids.to(torch.int32), "top_logprobs": logp.gather(1, ids)}


def work(case):
    op = case["op"]
    size = 4 if case["dtype"] == "fp32" else 2
    if op == "norm":
        T, D = case["tokens"], case["features"]
        per = 2 + 1 + (4 if case["residual"] else 0)
        return {"bytes": T * D * per + 2 * D + 4 * T * _blocks(D), "flops": 8 * T * D}
    if op == "gated":
        T, D = case["tokens"], case["features"]
        return {"bytes": T * D * 5 + 4 * T * _blocks(D), "flops": 8 * T * D}
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        scales = 4 * _blocks(K) * (M + _blocks(N))
        return {"bytes": M * K + N * K + size * M * N + scales, "flops": 2 * M * N * K}
    T, V, k = case["tokens"], case["vocab"], case["top"]
    return {"bytes": T * V * size + T * (8 + 4 + 4 + 8 * k), "flops": 6 * T * V}


def exact(case, seed):
    """The definitions in 64 bits, block by block of 128; e4m3 values as they are before their rounding."""
    st = prepare(case, seed)
    op = case["op"]

    def by_block(y):
        q, s = torch.empty_like(y), torch.empty((_blocks(y.shape[1]), y.shape[0]), dtype=torch.float64, device="cuda")
        for b in range(s.shape[0]):
            part = y[:, b * BLOCK:(b + 1) * BLOCK]
            s[b] = torch.clamp(part.abs().max(dim=1).values / E4M3_MAX, min=SCALE_MIN)
            q[:, b * BLOCK:(b + 1) * BLOCK] = part / s[b][:, None]
        return {"q": q, "scales": s}

    if op == "norm":
        h = st["x"].double() if st["residual"] is None else st["x"].double() + st["residual"].double()
        out = by_block(h / torch.sqrt(torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / h.shape[1] + st["eps"])
                       * st["weight"].double())
        if st["residual"] is not None:
            out["h"] = h
        return out
    if op == "gated":
        D = case["features"]
        gate = st["x"][:, :D].double()
        return by_block(gate * torch.special.expit(gate) * st["x"][:, D:].double())
    if op == "product":
        N, K = st["w"].shape
        y = torch.zeros((st["x"].shape[0], N), dtype=torch.float64, device="cuda")
        for b in range(_blocks(K)):
            cut = slice(b * BLOCK, (b + 1) * BLOCK)
            part = st["x"][:, cut].double() @ st["w"][:, cut].double().t()
            per_column = st["w_scales"][:, b].double()[torch.arange(N, device="cuda") // BLOCK]
            y += part * st["x_scales"][b].double()[:, None] * per_column[None, :]
        return y
    logp = torch.log_softmax(st["logits"].double(), dim=1)
    entropy = -torch.special.xlogy(logp.exp(), logp.exp()).sum(dim=1)
    order = torch.sort(st["logits"].float(), dim=1, descending=True, stable=True).indices[:, :case["top"]]
    return {"logprobs": logp.gather(1, st["tokens"][:, None])[:, 0], "entropy": entropy,
            "top_ids": order.to(torch.int32), "top_logprobs": logp.gather(1, order)}
