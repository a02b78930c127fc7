"""fp64 NumPy definitions of the operators round attention: keys and values into a paged cache, attention of drafted tokens over
it, and the verification of drafts. Slow and plain: loops over tokens and heads, nothing shared with the kernels."""
import numpy as np


def rotate(x, position, inv_freq, interleaved):
    """One head's features turned by position * inv_freq."""
    x = np.array(x, dtype=np.float64)
    half = len(inv_freq)
    for i, f in enumerate(inv_freq):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        w = np.longdouble(int(position)) * np.longdouble(f)
        c, s = float(np.cos(w)), float(np.sin(w))
        x[a], x[b] = x[a] * c - x[b] * s, x[b] * c + x[a] * s
    return x


def rope_append(q, k, v, k_cache, v_cache, slots, positions, inv_freq, q_weight, k_weight, eps, interleaved):
    """(q_out, k_cache, v_cache) of [T][heads][D] arrays and [pages][page_size][heads][D] caches."""
    k_cache, v_cache = k_cache.copy(), v_cache.copy()
    page_size = k_cache.shape[1]

    def one(x, weight, t):
        if weight is not None:
            x = x / np.sqrt(np.mean(x * x) + eps) * weight
        return rotate(x, positions[t], inv_freq, interleaved) if inv_freq is not None else x
    out = None if q is None else np.stack([[one(x, q_weight, t) for x in q[t]] for t in range(len(k))]) if len(k) else q
    for t, slot in enumerate(slots):
        if slot >= 0:
            page, at = divmod(int(slot), page_size)
            for h in range(k.shape[1]):
                k_cache[page, at, h] = one(k[t, h], k_weight, t)
                v_cache[page, at, h] = v[t, h]
    return out, k_cache, v_cache


def tree_attention(q, k_cache, v_cache, page_table, starts, context, mask, scale):
    """(out [T][heads][D], lse [T][heads], spread [T][heads][D], size [T][heads]): spread is sum p |v| and size the largest
    scale sum |q| |k| of a place seen, which say how far roundings may carry. mask: bool [T][tokens of its sequence], or None."""
    T, H, D = q.shape
    group = H // k_cache.shape[2]
    out, spread = np.zeros((T, H, D)), np.zeros((T, H, D))
    lse, size = np.full((T, H), -np.inf), np.zeros((T, H))
    page_size = k_cache.shape[1]
    for b, c in enumerate(context):
        for t in range(starts[b], starts[b + 1]):
            i, n = t - starts[b], starts[b + 1] - starts[b]
            places = np.array([p for p in range(c + n) if p < c or (mask[t][p - c] if mask is not None else p - c <= i)], dtype=int)
            if not len(places):
                continue
            pages = page_table[b][places // page_size]
            for h in range(H):
                K, V = k_cache[pages, places % page_size, h // group], v_cache[pages, places % page_size, h // group]
                with np.errstate(invalid="ignore", over="ignore"):
                    s = scale * (K @ q[t, h])
                    top = s.max()
                    p = np.exp(s - top)
                    lse[t, h] = top + np.log(p.sum())
                    p = p / p.sum()
                    out[t, h] = p @ V
                    spread[t, h] = p @ np.abs(V)
                    size[t, h] = abs(scale) * (np.abs(K) @ np.abs(q[t, h])).max()
    return out, lse, spread, size


def verify(logits, tokens, parents, uniforms, final_uniform, draft_probs=None, temperature=1.0):
    """One sequence's walk: (path, p of the next token, margin). margin is the least relative distance between the two sides of a
    decision on the way; p is None where the walk ends at a row that has no distribution."""
    V = logits.shape[1]

    def target(row):
        x = logits[row].astype(np.float64)
        if np.isnan(x).any() or np.isposinf(x).any() or np.isneginf(x).all():
            return None
        if temperature == 0:
            p = np.zeros(V)
            p[int(np.argmax(x))] = 1
            return p
        p = np.exp((x - x.max()) / temperature)
        return p / p.sum()
    if not len(tokens) or not 0 <= temperature < np.inf:
        return [], None, np.inf
    node, path, margin = 0, [], np.inf
    p = target(0)
    for j in range(1, len(tokens)):
        if p is None:
            break
        if parents[j] != node or not 0 <= tokens[j] < V:
            continue
        q = draft_probs[node].astype(np.float64) if draft_probs is not None else np.eye(1, V, int(tokens[j]))[0]
        left, right = float(uniforms[j]) * q[tokens[j]], p[tokens[j]]
        if max(left, right) > 0:
            margin = min(margin, abs(left - right) / max(left, right))
        if left < right:
            node, p = j, target(j)
            path.append(j)
            continue
        rest = np.maximum(p - q, 0)
        if rest.sum() > 0:
            p = rest / rest.sum()
    return path, p, margin
