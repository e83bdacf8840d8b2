"""Rotary positions and attention over a paged cache in 64 bits, for the tests: the formulas of
santa.h, on the CPU, one step at a time."""
import math

import numpy as np
import torch


def frequencies(rot, base=10000.0, scaling="none", factor=1.0, low=1.0, high=4.0, original=8192):
    """(radians a position of each pair, amplitude)."""
    out = []
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        turns = original * f / (2 * math.pi)
        if scaling == "linear":
            f /= factor
        elif scaling == "bands":
            if turns < low:
                f /= factor
            elif turns < high:
                s = (turns - low) / (high - low)
                f = (1 - s) * f / factor + s * f
        elif scaling == "ramp":
            def index(n):
                return rot * math.log(original / (n * 2 * math.pi)) / (2 * math.log(base))
            a, b = max(math.floor(index(high)), 0), min(math.ceil(index(low)), rot - 1)
            b = max(b, a + 0.001)
            r = min(max((i - a) / (b - a), 0.0), 1.0)
            f = r * f / factor + (1 - r) * f
        out.append(f)
    return np.array(out), 0.1 * math.log(factor) + 1 if scaling == "ramp" else 1.0


def rotate(x, f, amplitude, layout, pos):
    """float64 [B, T, H, d]: rows x (any tensor) at positions pos[b] + t."""
    x = x.double().cpu().numpy()
    rot = 2 * len(f)
    a = (np.asarray(pos, dtype=np.float64)[:, None] + np.arange(x.shape[1]))[..., None] * f
    c, s = amplitude * np.cos(a)[:, :, None], amplitude * np.sin(a)[:, :, None]
    out = x.copy()
    i = np.arange(rot // 2)
    u, v = (i, i + rot // 2) if layout == "halves" else (2 * i, 2 * i + 1)
    out[..., u] = x[..., u] * c - x[..., v] * s
    out[..., v] = x[..., u] * s + x[..., v] * c
    return out


def gather(pool, table, b, n):
    """Rows 0 .. n - 1 of sequence b: float64 [H_kv, n, d]; a page outside the pool holds zeros."""
    pool, page = pool.double().cpu().numpy(), pool.shape[2]
    out = np.zeros((pool.shape[1], n, pool.shape[3]))
    for j in range(n):
        p = int(table[b, j // page])
        if 0 <= p < pool.shape[0]:
            out[:, j] = pool[p, :, j % page]
    return out


def attention(q, k, v, table, pos, counts=None, window=0, sinks=0, scale=0.0):
    """float64 [B, T, H_q, d], rows that are not live zero, and the weighted distance of the values
    from the result, sum_j p_j |v_j - o|; k and v pools [n_pages, H_kv, page, d].  A key of weight 0
    adds nothing, whatever its value."""
    q = q.double().cpu().numpy()
    B, T, H_q, d = q.shape
    H_kv = k.shape[1]
    sigma = float(np.float32(scale)) if scale else 1.0 / math.sqrt(d)
    out, spread = np.zeros((B, T, H_q, d)), np.zeros((B, T, H_q, d))
    with np.errstate(invalid="ignore"):
        for b in range(B):
            n = T if counts is None else int(counts[b])
            p0 = int(pos[b])
            if n == 0:
                continue
            kb, vb = gather(k, table, b, p0 + n), gather(v, table, b, p0 + n)
            for t in range(n):
                j = np.arange(p0 + t + 1)
                if window:
                    j = j[(j > p0 + t - window) | (j < sinks)]
                s = np.einsum("hgd,hnd->hgn", q[b, t].reshape(H_kv, -1, d), kb[:, j]) * sigma
                w = np.exp(s - s.max(-1, keepdims=True))
                w /= w.sum(-1, keepdims=True)
                o = np.einsum("hgn,hnd->hgd", w, vb[:, j])
                out[b, t] = o.reshape(H_q, d)
                spread[b, t] = np.stack([np.einsum("gn,ngd->gd", w[h], np.abs(vb[h, j][:, None] - o[h][None]))
                                         for h in range(H_kv)]).reshape(H_q, d)
    return out, spread


# A bf16 rounding is off by half a step, 2^-8 of the value.  The result has one.  Each weight has one,
# e_j, in the sum over V and in the sum of weights alike, so that it moves the result by sum p_j e_j
# (v_j - o) / (1 + sum p_j e_j).  Scores are fp32 sums of d products, off by d steps of 2^-24 of
# their size at most, exponentials by 2^-21: together 2^-10 of a weight for scores up to 2^6.
def tolerance(out, spread):
    return 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + 2.0 ** -10) * 1.01 * spread + 2.0 ** -22 * np.nanmax(np.abs(out), initial=0.0)


def pages(gen, lengths, page, columns, spare=2):
    """(table [B, columns], n_pages): pages in no order, entries that no key needs name none."""
    need = [-(-n // page) for n in lengths]
    n_pages = sum(need) + spare
    perm = torch.randperm(n_pages, generator=gen)
    table = torch.full((len(lengths), columns), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n].to(torch.int32)
        at += n
    return table, n_pages
