"""Plain fp64 implementations of the 8-bit row operators: e4m3 codes, RMS norm with the residual's
addition, the gated activation, the block-scaled product, and log probabilities with entropy and top
tokens. NumPy only; shares no code with the GPU path."""
from __future__ import annotations

import numpy as np

BLOCK = 128
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126


def _e4m3_table() -> np.ndarray:
    """The value of each of the 256 e4m3 codes: sign, 4 exponent bits (bias 7), 3 mantissa bits, no
    infinities, NaN at all ones."""
    t = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        t[c] = np.nan if (c & 127) == 127 else (-v if c & 128 else v)
    return t


E4M3 = _e4m3_table()


def decode_e4m3(codes: np.ndarray) -> np.ndarray:
    return E4M3[codes]


def e4m3_step(v: np.ndarray) -> np.ndarray:
    """The distance between neighbouring e4m3 values around |v| (v up to 448)."""
    a = np.maximum(np.abs(v), 2.0 ** -6)
    return 2.0 ** (np.floor(np.log2(a)) - 3)


def encode_e4m3(v: np.ndarray) -> np.ndarray:
    """Nearest e4m3 code (ties to the even mantissa, past 448: 448, NaN to NaN)."""
    pos = E4M3[:127]
    a = np.abs(v)
    hi = np.clip(np.searchsorted(pos, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    c = np.where(a >= E4M3_MAX, 126, c)
    c = np.where(np.isnan(v), 127, c)
    return (c | (np.signbit(v).astype(np.int64) << 7)).astype(np.uint8)


def block_scales(y: np.ndarray) -> np.ndarray:
    """[ceil(D/128)][T] scales of y [T][D]; NaN does not take part."""
    T, D = y.shape
    nb = -(-D // BLOCK)
    s = np.empty((nb, T))
    for b in range(nb):
        a = np.abs(y[:, b * BLOCK:(b + 1) * BLOCK])
        s[b] = np.maximum(np.where(np.isnan(a), 0.0, a).max(axis=1) / E4M3_MAX, SCALE_MIN)
    return s


def spread(scales: np.ndarray, D: int) -> np.ndarray:
    """[T][D]: each element's scale."""
    return np.repeat(scales.T, BLOCK, axis=1)[:, :D]


def add_rmsnorm(x, weight, residual=None, eps=1e-6):
    """(h, y) in fp64."""
    h = x.astype(np.float64) if residual is None else x.astype(np.float64) + residual.astype(np.float64)
    with np.errstate(all="ignore"):
        y = h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps) * weight.astype(np.float64)
    return h, y


def silu_mul(x):
    D = x.shape[1] // 2
    g, u = x[:, :D].astype(np.float64), x[:, D:].astype(np.float64)
    with np.errstate(all="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def block_mm(xq, x_scales, wq, w_scales):
    """(Y, sum of the terms' magnitudes) of e4m3 codes xq [M][K], wq [N][K] and their scales."""
    N = wq.shape[0]
    y, mag = 0.0, 0.0
    with np.errstate(all="ignore"):
        for b in range(x_scales.shape[0]):
            cut = slice(b * BLOCK, (b + 1) * BLOCK)
            xv, wv = decode_e4m3(xq[:, cut]), decode_e4m3(wq[:, cut])
            f = x_scales[b].astype(np.float64)[:, None] * w_scales[:, b].astype(np.float64)[np.arange(N) // BLOCK][None, :]
            y = y + (xv @ wv.T) * f
            mag = mag + (np.abs(xv) @ np.abs(wv).T) * np.abs(f)
    return y, mag


def token_logprobs(logits, tokens, k):
    """(logprobs, entropy, top_ids, top_logprobs) of fp64 logits, row by row from the definitions."""
    T, V = logits.shape
    lp, ent = np.full(T, np.nan), np.zeros(T)
    ids, tlp = np.full((T, k), -1, dtype=np.int64), np.full((T, k), -np.inf)
    for t in range(T):
        x = logits[t].astype(np.float64)
        order = [i for i in np.argsort(np.where(np.isnan(x), np.inf, -x), kind="stable") if x[i] > -np.inf][:k]
        ids[t, :len(order)] = order
        if np.isnan(x).any() or (x == np.inf).any():
            ent[t], tlp[t] = np.nan, np.nan
            continue
        if (x == -np.inf).all():
            logp = x
        else:
            d = x - x.max()
            logp = d - np.log(np.exp(d).sum())
            live = np.exp(logp) > 0
            ent[t] = -(np.exp(logp[live]) * logp[live]).sum()
        tlp[t, :len(order)] = logp[order]
        if 0 <= tokens[t] < V:
            lp[t] = logp[tokens[t]]
    return lp, ent, ids, tlp
