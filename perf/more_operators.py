"""The operators of one speculative decoding step beside the products, each as one measured pass.

  append    a projection's queries, keys and values: RMS norm of each query and key head, rotation by position,
            keys and values written to their slots of a paged cache
  attention of drafted tokens over a paged cache: token i of a sequence sees the sequence's context and those
            of its drafted tokens that its mask names (without masks: the ones before it and itself)
  verify    the drafted tokens held against the target's probabilities with given random numbers: how many are
            kept, which, and the token that follows them

`run` computes them with elementary torch operations in 32 bits (angles and sums over the vocabulary in 64) or,
with `own`, through the package.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # one token of one sequence being decoded
        {"name": "append_1_bf16", "op": "append", "tokens": 1, "q_heads": 32, "kv_heads": 8, "dim": 128, "rot": 128, "interleaved": False, "norm": True, "page": 16, "dtype": "bf16"},
        # a ragged decode batch of a model with small heads, partly rotated in neighbouring pairs, without norms
        {"name": "append_333_fp16", "op": "append", "tokens": 333, "q_heads": 14, "kv_heads": 2, "dim": 80, "rot": 32, "interleaved": True, "norm": False, "page": 48, "dtype": "fp16"},
        # a chunk of a long prompt
        {"name": "append_8192_bf16", "op": "append", "tokens": 8192, "q_heads": 32, "kv_heads": 8, "dim": 128, "rot": 128, "interleaved": False, "norm": True, "page": 64, "dtype": "bf16"},
        # one token of one sequence after a short prompt
        {"name": "attention_1x1_600_bf16", "op": "attention", "batch": 1, "tokens": 1, "context_lo": 600, "context_hi": 600, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 16, "tree": False, "lse": False, "dtype": "bf16"},
        # a decode batch without drafts
        {"name": "attention_64x1_16k_bf16", "op": "attention", "batch": 64, "tokens": 1, "context_lo": 500, "context_hi": 16000, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 16, "tree": False, "lse": False, "dtype": "bf16"},
        # short chains of drafts, small heads, seven queries to a key, pages that no tile divides
        {"name": "attention_23x5_3k_fp16", "op": "attention", "batch": 23, "tokens": 5, "context_lo": 0, "context_hi": 3001, "q_heads": 14, "kv_heads": 2, "dim": 64, "page": 48, "tree": False, "lse": True, "dtype": "fp16"},
        # a batch of drafted trees
        {"name": "attention_16x32_8k_bf16", "op": "attention", "batch": 16, "tokens": 32, "context_lo": 1000, "context_hi": 8000, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "tree": True, "lse": False, "dtype": "bf16"},
        # a large tree over one long document
        {"name": "attention_1x64_128k_bf16", "op": "attention", "batch": 1, "tokens": 64, "context_lo": 131000, "context_hi": 131000, "q_heads": 64, "kv_heads": 8, "dim": 128, "page": 64, "tree": True, "lse": True, "dtype": "bf16"},
        # one sequence with a chain of four drafts from a small model
        {"name": "verify_1x5_32k_fp32", "op": "verify", "batch": 1, "tokens": 5, "vocab": 32001, "tree": False, "probs": True, "greedy": False, "dtype": "fp32"},
        # a batch of trees drafted without probabilities, some sequences greedy
        {"name": "verify_32x16_128k_bf16", "op": "verify", "batch": 32, "tokens": 16, "vocab": 131072, "tree": True, "probs": False, "greedy": True, "dtype": "bf16"},
        # a large batch with short chains
        {"name": "verify_192x6_128k_bf16", "op": "verify", "batch": 192, "tokens": 6, "vocab": 131072, "tree": False, "probs": True, "greedy": False, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "verify"])
    dtype = rng.choice(["bf16", "fp16"])
    kv_heads = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 48, 64, 128])
    if op == "append":
        q_heads = kv_heads * rng.choice([1, 2, 3, 4, 7, 8])
        dim = rng.choice([64, 80, 96, 128, 192, 256])
        rot = rng.choice([dim, dim, dim // 2 // 16 * 16, 32])
        tokens = _log_int(rng, 1, max(1, min(16384, 8192 * 48 * 128 // ((q_heads + 2 * kv_heads) * dim))))
        return {"op": op, "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "rot": rot,
                "interleaved": rng.random() < 0.3, "norm": rng.random() < 0.6, "page": page, "dtype": dtype}
    if op == "attention":
        group = rng.choice([1, 2, 4, 4, 7, 8, 16])
        dim = rng.choice([64, 64, 80, 96, 128, 128, 128, 192, 256])
        tokens = rng.choice([1, 1, 1, rng.randint(2, 9), rng.randint(8, 33), rng.randint(16, 80)])
        batch = _log_int(rng, 1, 200)
        # no more than the largest listed cases read (64 sequences of 8250 on average) and multiply (64 tokens by 131000)
        most = min(64 * 8250 * 8 * 128 // (batch * kv_heads * dim), 64 * 131000 * 64 * 128 // (batch * tokens * kv_heads * group * dim))
        hi = _log_int(rng, 1, max(1, min(131072, most - tokens)))
        return {"op": op, "batch": batch, "tokens": tokens, "context_lo": rng.choice([0, hi // 8, hi]), "context_hi": hi,
                "q_heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim, "page": page,
                "tree": tokens > 2 and rng.random() < 0.7, "lse": rng.random() < 0.4, "dtype": dtype}
    vocab = _log_int(rng, 1000, 160000)
    tokens = rng.randint(1, 17)
    batch = _log_int(rng, 1, max(1, min(256, 192 * 6 * 131072 // (tokens * vocab))))
    return {"op": op, "batch": batch, "tokens": tokens, "vocab": vocab, "tree": rng.random() < 0.5, "probs": rng.random() < 0.5,
            "greedy": rng.random() < 0.4, "dtype": rng.choice(["bf16", "fp16", "fp32"])}


def _spread(lo, hi, n):
    return [lo + (hi - lo) * i // max(1, n - 1) if n > 1 else hi for i in range(n)]


def _counts(case):
    """Drafted tokens of each sequence, the last token kept included: up to two fewer than the most."""
    return [max(1, case["tokens"] - i % 3) for i in range(case["batch"])]


def _parents(n, tree, rng):
    """The parent of each drafted token of a sequence, -1 for the first."""
    return [-1 if i == 0 else rng.randint(max(0, i - 1 - i // 2), i - 1) if tree else i - 1 for i in range(n)]


def _masks(parents):
    """64-bit words of each token: bit j of word j // 64 where the token is j or descends from it."""
    words = (len(parents) + 63) // 64
    seen = []
    for i, p in enumerate(parents):
        seen.append((seen[p] if p >= 0 else 0) | 1 << i)
    out = [[s >> (64 * w) & (1 << 64) - 1 for w in range(words)] for s in seen]
    return [[v - (1 << 64) if v >> 63 else v for v in row] for row in out]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = random.Random(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def numbers(values, dtype):
        return torch.tensor(values, dtype=dtype, device="cuda")

    st = {"case": case}
    if op == "append":
        T, Hq, Hk, D, R = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"], case["rot"]
        # the rows of one projection; a few features of the keys are much larger than the others
        rows = normal(T, Hq + 2 * Hk, D) * torch.where(torch.rand(D, generator=g, device="cuda") < 0.03, 6.0, 1.0)
        st["rows"] = rows.to(dt)
        st["q_weight"] = (1.0 + 0.2 * normal(D)).to(dt) if case["norm"] else None
        st["k_weight"] = (1.0 + 0.2 * normal(D)).to(dt) if case["norm"] else None
        st["inv_freq"] = 5e5 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float32) / R)
        first = rng.randint(0, 131072)
        st["positions"] = first + torch.arange(T, device="cuda", dtype=torch.int64)
        pages = -(-T // case["page"]) + 3
        st["k_cache"] = normal(pages, case["page"], Hk, D).to(dt)
        st["v_cache"] = normal(pages, case["page"], Hk, D).to(dt)
        order = torch.randperm(pages, generator=g, device="cuda")
        at = rng.randint(0, case["page"]) + torch.arange(T, device="cuda")
        st["slots"] = order[at // case["page"]] * case["page"] + at % case["page"]
        st["q_out"] = torch.empty((T, Hq, D), dtype=dt, device="cuda")
    elif op == "attention":
        B, Hq, Hk, D, page = case["batch"], case["q_heads"], case["kv_heads"], case["dim"], case["page"]
        contexts, counts = _spread(case["context_lo"], case["context_hi"], B), _counts(case)
        rng.shuffle(contexts)
        T = sum(counts)
        starts = [0]
        for n in counts:
            starts.append(starts[-1] + n)
        need = [-(-(c + n) // page) for c, n in zip(contexts, counts)]
        pages = sum(need)
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).tolist()
        table, at = [], 0
        for n in need:
            table.append(order[at:at + n] + [0] * (max(need) - n))
            at += n
        st["k_cache"], st["v_cache"] = (torch.empty((pages, page, Hk, D), dtype=dt, device="cuda") for _ in "kv")
        spread = torch.exp(0.3 * normal(D))
        st["k_cache"].copy_(normal(pages, page, Hk, D) * spread)
        st["v_cache"].copy_(normal(pages, page, Hk, D) + 0.3 * normal(D))
        st["q"] = (1.5 * normal(T, Hq, D)).to(dt)
        st["table"], st["starts"], st["context"] = (numbers(v, torch.int32) for v in (table, starts, contexts))
        words = (case["tokens"] + 63) // 64
        st["mask"] = None
        if case["tree"]:
            rows = [r + [0] * (words - len(r)) for n in counts for r in _masks(_parents(n, True, rng))]
            st["mask"] = numbers(rows, torch.int64)
        st["out"] = torch.empty((T, Hq, D), dtype=dt, device="cuda")
        st["lse"] = torch.empty((T, Hq), dtype=torch.float32, device="cuda") if case["lse"] else None
    else:
        B, V, counts = case["batch"], case["vocab"], _counts(case)
        T = sum(counts)
        starts = [0]
        for n in counts:
            starts.append(starts[-1] + n)
        parents = [p for n in counts for p in _parents(n, case["tree"], rng)]
        above = numbers([max(p, 0) + s for s, n in zip(starts, counts) for p in parents[s:s + n]], torch.int64)
        # the head's logits: a broad body and some tens of tokens that the context favours
        x = normal(T, V) * 2.0
        x.scatter_add_(1, torch.randint(0, V, (T, 40), generator=g, device="cuda"), 8.0 + 3.0 * normal(T, 40))
        st["logits"] = x.to(dt)
        cool = [0.0 if case["greedy"] and b % 3 == 0 else (0.7, 1.0, 0.85, 1.3)[b % 4] for b in range(B)]
        st["temperature"] = numbers(cool, torch.float32)
        # a smaller model's guess at the same distributions; a child is drawn from its parent's row
        x = x.add_(normal(T, V), alpha=0.7)
        if case["probs"]:
            st["draft_probs"] = torch.softmax(x, dim=1)
            drawn = torch.multinomial(st["draft_probs"], 16, replacement=True, generator=g)
        else:
            st["draft_probs"] = None
            drawn = torch.topk(x, 16, dim=1).indices
        rank, children = [], {}
        for p in above.tolist():
            children[p] = children.get(p, -1) + 1
            rank.append(children[p] % 16)
        st["tokens"] = drawn[above, numbers(rank, torch.int64)]
        st["parents"], st["starts"] = numbers(parents, torch.int32), numbers(starts, torch.int32)
        st["uniforms"] = torch.rand(T, generator=g, device="cuda")
        st["final_uniforms"] = torch.rand(B, generator=g, device="cuda")
        st["accepted"] = torch.empty(B, dtype=torch.int32, device="cuda")
        st["path"] = torch.empty((B, max(1, case["tokens"] - 1)), dtype=torch.int32, device="cuda")
        st["next_tokens"] = torch.empty(B, dtype=torch.int64, device="cuda")
    return st


def _run_own(st):
    import weight_only_quantized_wq4_gb300 as wq4
    case = st["case"]
    if case["op"] == "append":
        Hq, Hk = case["q_heads"], case["kv_heads"]
        rows = st["rows"]
        wq4.rope_append(rows[:, :Hq], rows[:, Hq:Hq + Hk], rows[:, Hq + Hk:], st["k_cache"], st["v_cache"], st["slots"],
                        st["positions"], st["inv_freq"], q_weight=st["q_weight"], k_weight=st["k_weight"], eps=EPS,
                        interleaved=case["interleaved"], q_out=st["q_out"])
        return {"q": st["q_out"], "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
    if case["op"] == "attention":
        if "workspace" not in st:
            st["workspace"] = wq4.alloc_workspace(wq4.tree_attention_workspace_bytes(
                case["batch"], case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]))
        wq4.tree_attention(st["q"], st["k_cache"], st["v_cache"], st["table"], st["starts"], st["context"],
                           max_tokens=case["tokens"], mask=st["mask"], out=st["out"], lse=st["lse"], workspace=st["workspace"])
        return {"out": st["out"], "lse": st["lse"]} if case["lse"] else {"out": st["out"]}
    wq4.verify_drafts(st["logits"], st["tokens"], st["parents"], st["starts"], st["uniforms"], st["final_uniforms"],
                      max_tokens=case["tokens"], draft_probs=st["draft_probs"], temperature=st["temperature"],
                      accepted=st["accepted"], path=st["path"], next_tokens=st["next_tokens"])
    return {"accepted": st["accepted"], "path": st["path"], "next_tokens": st["next_tokens"]}


def _rotated(x, angles, interleaved):
    """x [T][heads][D] with its first 2 angles.shape[1] features rotated, in 32 bits."""
    R = 2 * angles.shape[1]
    cos, sin = torch.cos(angles).float()[:, None], torch.sin(angles).float()[:, None]
    if interleaved:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((turned, x[..., R:]), dim=-1)


def _append(st):
    case, dt = st["case"], DTYPES[st["case"]["dtype"]]
    Hq, Hk, D = case["q_heads"], case["kv_heads"], case["dim"]
    q, k, v = st["rows"][:, :Hq].float(), st["rows"][:, Hq:Hq + Hk].float(), st["rows"][:, Hq + Hk:]
    if case["norm"]:
        q = q * torch.rsqrt((q * q).mean(dim=-1, keepdim=True) + EPS) * st["q_weight"].float()
        k = k * torch.rsqrt((k * k).mean(dim=-1, keepdim=True) + EPS) * st["k_weight"].float()
    angles = st["positions"].double()[:, None] * st["inv_freq"].double()
    st["q_out"].copy_(_rotated(q, angles, case["interleaved"]))
    st["k_cache"].view(-1, Hk, D)[st["slots"]] = _rotated(k, angles, case["interleaved"]).to(dt)
    st["v_cache"].view(-1, Hk, D)[st["slots"]] = v
    return {"q": st["q_out"], "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _attention(st):
    case, dt = st["case"], DTYPES[st["case"]["dtype"]]
    B, n, Hq, Hk, D, page = case["batch"], case["tokens"], case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    dev, T = st["q"].device, st["q"].shape[0]
    starts, context = st["starts"].long(), st["context"].long()
    count = starts[1:] - starts[:-1]
    L = st["table"].shape[1] * page
    pos = torch.arange(L, device=dev)
    pages = st["table"].long()[:, pos // page]
    k = st["k_cache"][pages, pos % page].permute(0, 2, 3, 1).float()             # [B][Hk][D][L]
    v = st["v_cache"][pages, pos % page].permute(0, 2, 1, 3).float()             # [B][Hk][L][D]
    i = torch.arange(n, device=dev)
    row = (starts[:-1, None] + i).clamp_max(T - 1)                               # [B][n]
    q = st["q"][row].float().view(B, n, Hk, Hq // Hk, D).transpose(1, 2).reshape(B, Hk, -1, D)
    j = pos[None] - context[:, None]                                             # [B][L]: the drafted token at a position
    if st["mask"] is None:
        drafted = j[:, None] <= i[None, :, None]
    else:
        words = st["mask"][row]                                                  # [B][n][words]
        at = j.clamp(0, 64 * words.shape[2] - 1)[:, None].expand(B, n, L)
        drafted = (words.gather(2, at // 64) >> at % 64 & 1) != 0
    sees = torch.where(j[:, None] < 0, True, drafted & (j < count[:, None])[:, None])   # [B][n][L]
    sees = sees[:, None, :, None].expand(B, 1, n, Hq // Hk, L).reshape(B, 1, -1, L)
    s = torch.where(sees, q @ k * (1.0 / math.sqrt(D)), -math.inf)
    top = s.amax(dim=-1, keepdim=True)
    p = torch.exp(s - torch.where(top > -math.inf, top, 0.0))
    z = p.sum(dim=-1, keepdim=True)
    o = torch.where(z > 0, p @ v / z, 0.0)
    lse = (top + torch.log(z))[..., 0]
    kept = (i[None] < count[:, None])[:, :, None]                                # rows of the shorter sequences drop out
    o = o.view(B, Hk, n, -1, D).transpose(1, 2).reshape(B, n, Hq, D)
    out = {"out": o[kept[:, :, 0]].to(dt)}
    if case["lse"]:
        out["lse"] = lse.view(B, Hk, n, -1).transpose(1, 2).reshape(B, n, Hq)[kept[:, :, 0]]
    return out


def _verify(st):
    case = st["case"]
    B, n, V = case["batch"], case["tokens"], case["vocab"]
    starts, dev = st["starts"].long(), st["logits"].device
    count, base = starts[1:] - starts[:-1], starts[:-1]
    every = torch.arange(B, device=dev)
    greedy = (st["temperature"] == 0)[:, None]
    heat = 1.0 / torch.where(greedy[:, 0], 1.0, st["temperature"])[:, None]

    def weights(row):
        """exp(x - max) of the rows' scaled logits; for greedy sequences 1 at the first largest and 0 elsewhere."""
        x = st["logits"][row].float()
        first = torch.zeros_like(x).scatter_(1, x.argmax(dim=1, keepdim=True), 1.0)
        x = x * heat
        w = torch.where(greedy, first, torch.exp(x - x.amax(dim=1, keepdim=True)))
        return w, w.sum(dim=1, dtype=torch.float64)

    node = torch.zeros(B, dtype=torch.int64, device=dev)
    accepted = torch.zeros(B, dtype=torch.int64, device=dev)
    path = torch.full((B, max(1, n - 1) + 1), -1, dtype=torch.int32, device=dev)  # (the last column takes what is not kept)
    w, z = weights(base)
    for j in range(1, n):
        row = (base + j).clamp_max(st["tokens"].shape[0] - 1)
        token = st["tokens"][row]
        tried = (j < count) & (st["parents"][row].long() == node)
        q = torch.ones(B, device=dev) if st["draft_probs"] is None else st["draft_probs"][base + node, token]
        kept = tried & (st["uniforms"][row].double() * q.double() * z < w[every, token].double())
        # not kept: what the draft's distribution leaves of the target's
        if st["draft_probs"] is None:
            left = w.scatter(1, token[:, None], 0.0)
        else:
            left = (w * (1.0 / z).float()[:, None] - st["draft_probs"][base + node]).clamp_min(0.0)
        z_left = left.sum(dim=1, dtype=torch.float64)
        lost = tried & ~kept & (z_left > 0)
        next_w, next_z = weights(row)
        w = torch.where(kept[:, None], next_w, torch.where(lost[:, None], left, w))
        z = torch.where(kept, next_z, torch.where(lost, z_left, z))
        path[every, torch.where(kept, accepted, path.shape[1] - 1)] = j
        accepted += kept
        node = torch.where(kept, j, node)
    upto = torch.cumsum(w.double(), dim=1)
    aim = (st["final_uniforms"].double() * z)[:, None]
    following = (upto > aim).to(torch.int8).argmax(dim=1)
    return {"accepted": accepted.to(torch.int32), "path": path[:, :-1], "next_tokens": following}


def run(st):
    if own:
        return _run_own(st)
    return {"append": _append, "attention": _attention, "verify": _verify}[st["case"]["op"]](st)


def work(case):
    op, size = case["op"], 4 if case["dtype"] == "fp32" else 2
    if op == "append":
        T, heads, D = case["tokens"], case["q_heads"] + 2 * case["kv_heads"], case["dim"]
        return {"bytes": 4 * T * heads * D + 16 * T, "flops": 8 * T * heads * D}
    if op == "attention":
        counts, contexts = _counts(case), _spread(case["context_lo"], case["context_hi"], case["batch"])
        seen = sum(contexts) + sum(counts)
        mean = sum(contexts) / len(contexts)
        rows = sum(counts) * case["q_heads"] * case["dim"]
        return {"bytes": 2 * size * seen * case["kv_heads"] * case["dim"] + 2 * size * rows,
                "flops": 4 * rows * (mean + case["tokens"] / 2)}
    # the rows that a walk comes to: about 0.7 of the drafts tried are kept; and the draft's row where it stops
    counts = _counts(case)
    visited = sum((1 - 0.7 ** n) / 0.3 for n in counts)
    probs = 4 * case["vocab"] * case["batch"] * 0.7 if case["probs"] and case["tokens"] > 1 else 0
    return {"bytes": visited * case["vocab"] * size + probs, "flops": 6 * visited * case["vocab"]}


def exact(case, seed):
    """The definitions in 64 bits, sequence by sequence; no value for the whole numbers of a verification."""
    if case["op"] == "verify":
        return None
    st = prepare(case, seed)
    if case["op"] == "append":
        T, Hq, Hk, R = case["tokens"], case["q_heads"], case["kv_heads"], case["rot"]
        angle = st["positions"].double().view(T, 1) * st["inv_freq"].double().view(1, -1)
        turn = torch.polar(torch.ones_like(angle), angle).view(T, 1, R // 2)

        def turned(x, weight):
            x = x.double()
            if case["norm"]:
                x = x / torch.sqrt(torch.linalg.vector_norm(x, dim=2, keepdim=True) ** 2 / x.shape[2] + EPS) * weight.double()
            pairs = x[:, :, :R].reshape(T, -1, R // 2, 2) if case["interleaved"] else x[:, :, :R].reshape(T, -1, 2, R // 2).transpose(2, 3)
            pairs = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            pairs = pairs if case["interleaved"] else pairs.transpose(2, 3)
            return torch.cat((pairs.reshape(T, -1, R), x[:, :, R:]), dim=2)

        k_cache, v_cache = st["k_cache"].double(), st["v_cache"].double()
        page, offset = st["slots"] // case["page"], st["slots"] % case["page"]
        k_cache[page, offset] = turned(st["rows"][:, Hq:Hq + Hk], st["k_weight"])
        v_cache[page, offset] = st["rows"][:, Hq + Hk:].double()
        return {"q": turned(st["rows"][:, :Hq], st["q_weight"]), "k_cache": k_cache, "v_cache": v_cache}
    starts, contexts = st["starts"].tolist(), st["context"].tolist()
    group = case["q_heads"] // case["kv_heads"]
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(st["q"].shape[:2], dtype=torch.float64, device="cuda")
    for b, c in enumerate(contexts):
        lo, hi = starts[b], starts[b + 1]
        n, used = hi - lo, -(-(c + hi - lo) // case["page"])
        pages = st["table"][b, :used].long()
        k, v = (st[x][pages].flatten(0, 1)[:c + n].double() for x in ("k_cache", "v_cache"))
        hidden = torch.triu(torch.ones(n, n, dtype=torch.bool, device="cuda"), diagonal=1)
        if st["mask"] is not None:
            words = st["mask"][lo:hi].cpu().tolist()
            hidden = torch.tensor([[not w[j // 64] >> j % 64 & 1 for j in range(n)] for w in words], device="cuda")
        for h in range(case["q_heads"]):
            s = st["q"][lo:hi, h].double() @ k[:, h // group].t() / math.sqrt(case["dim"])
            s[:, c:].masked_fill_(hidden, -math.inf)
            lse[lo:hi, h] = torch.logsumexp(s, dim=1)
            out[lo:hi, h] = torch.softmax(s, dim=1) @ v[:, h // group]
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}
