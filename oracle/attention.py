"""The attention step in fp64, from its formulas: head norms, rotary positions, e4m3 quantisation and causal
attention over cached rows. numpy loops over sequences and heads; nothing here knows of pages, tiles or streams."""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
AMAX_MIN = 2.0 ** -60


def e4m3_values() -> np.ndarray:
    """The 127 values of the non-negative finite codes 0 .. 126."""
    code = np.arange(127)
    e, m = code >> 3, code & 7
    return np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))


def norm_heads(x: np.ndarray, w, eps: float) -> np.ndarray:
    """x [..., hd] / sqrt(mean(x^2) + eps) * w."""
    return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * w


def rotate(x: np.ndarray, pos: np.ndarray, freq, interleaved: bool, mscale: float = 1.0) -> np.ndarray:
    """The first 2 len(freq) elements of each head of x [T, H, hd] turned by pos * freq radians."""
    y = x.copy()
    half = len(freq)
    for i, f in enumerate(freq):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = np.cos(pos * float(f))[:, None] * mscale, np.sin(pos * float(f))[:, None] * mscale
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def row_scale(x: np.ndarray) -> np.ndarray:
    return np.maximum(np.abs(x).max(-1), AMAX_MIN) / E4M3_MAX


def seen_keys(position: int, window=None, sinks: int = 0) -> np.ndarray:
    """The keys that the token at `position` sees: all up to its own, or, with a window, the first `sinks` ones and the last
    `window` ones."""
    j = np.arange(position + 1)
    return j if window is None else j[(j < sinks) | (j > position - window)]


def attention(q, keys, values, starts, group: int, scale: float, window=None, sinks: int = 0) -> tuple:
    """q [T, Hq, hd]; keys, values: for each sequence [L, Hkv, hd]; its queries are rows starts[s] .. starts[s + 1] - 1
    and its last positions. Returns the output [T, Hq, hd] and two bounds' ingredients of each element or row:
    sum_j p_j |v_j| and max_j scale sum_i |q_i k_ji|. Rows of no sequence, or with no key, are zero."""
    T, hq, hd = q.shape
    out, weight, size = np.zeros((T, hq, hd)), np.zeros((T, hq, hd)), np.zeros((T, hq))
    for s, (k, v) in enumerate(zip(keys, values)):
        a, b = starts[s], starts[s + 1]
        for t in range(a, b):
            if len(k) - (b - a) + (t - a) < 0:
                continue
            seen = seen_keys(len(k) - (b - a) + (t - a), window, sinks)
            for h in range(hq):
                kk, vv = k[seen, h // group], v[seen, h // group]
                z = scale * (kk @ q[t, h])
                p = np.exp(z - z.max())
                p /= p.sum()
                out[t, h], weight[t, h] = p @ vv, p @ np.abs(vv)
                size[t, h] = scale * (np.abs(kk) @ np.abs(q[t, h])).max()
    return out, weight, size
