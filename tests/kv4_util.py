"""The 4-bit cache format and windowed attention in 64 bits, for the tests: the formulas of
santa.h, on the CPU, one step at a time."""
import math

import numpy as np
import torch

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# scale code -> value; 0xE2 (10240) is the largest the writer uses, 0xF8.. are not numbers
SCALE = np.array([(m * 2.0 ** -17 if e == 0 else (8 + m) * 2.0 ** (e - 18)) if e < 31 else math.nan
                  for e in range(32) for m in range(8)])
MAX_CODE = 0xE2


def nearest_even(values, table):
    """Index of the table entry nearest each value (table ascending), ties to the even index."""
    hi = np.clip(np.searchsorted(table, values), 1, len(table) - 1)
    lo = hi - 1
    a, b = values - table[lo], table[hi] - values
    return np.where((b < a) | ((b == a) & (hi % 2 == 0)), hi, lo)


def quantise(x: torch.Tensor):
    """bf16 [..., d] -> (codes [..., d/2], scales [..., d/16]) as uint8 arrays."""
    a = x.double().numpy()
    g = a.reshape(*a.shape[:-1], -1, 16)
    amax = np.abs(g).max(-1)
    bad = ~np.isfinite(amax)
    sc = nearest_even(np.where(bad, 0.0, amax) / 6.0, SCALE[:MAX_CODE + 1])
    s = SCALE[sc]
    live = (s > 0) & ~bad
    y = np.abs(np.where(bad[..., None], 0.0, g)) / np.where(live, s, 1.0)[..., None]
    idx = nearest_even(y, GRID) * live[..., None]
    code = (idx | np.where(np.signbit(g), 8, 0) * live[..., None]).reshape(a.shape).astype(np.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), np.where(bad, 0xFF, sc).astype(np.uint8)


def values(codes, scales):
    """float64 [..., d] that codes and scales (uint8 arrays) stand for."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    c = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1)
    v = GRID[c & 7] * np.where(c & 8, -1.0, 1.0)
    return v * np.repeat(SCALE[scales], 16, -1)


def visible(n, window, sinks):
    j = np.arange(n)
    return j if window == 0 else j[(j >= n - window) | (j < sinks)]


def attention(q, k, v, seq_lens, window=0, sinks=0, scale=0.0):
    """float64 [B, H_q, d]; q, k, v any tensors or arrays, k and v [B, H_kv, n, d]."""
    q, k, v = (np.asarray(x.double() if isinstance(x, torch.Tensor) else x, dtype=np.float64) for x in (q, k, v))
    B, H_q, d = q.shape
    H_kv = k.shape[1]
    out = np.zeros((B, H_q, d))
    sigma = float(np.float32(scale)) if scale else 1.0 / math.sqrt(d)
    for b in range(B):
        j = visible(int(seq_lens[b]), window, sinks)
        if len(j) == 0:
            continue
        for h in range(H_q):
            g = h // (H_q // H_kv)
            s = k[b, g][j] @ q[b, h] * sigma
            w = np.exp(s - s.max())
            out[b, h] = (w / w.sum()) @ v[b, g][j]
    return out
