"""Numerics of the windowed and 4-bit attention kernels at scores, weights and lengths where
fp32 arithmetic gives the answer and narrower steps on the way would not.

Scores here are sums with one product that is not zero, so that they are exact in fp32: what is
tested is what follows, the softmax and the weighted sum.
"""
import math

import numpy as np
import pytest
import torch

from stochastic_sparse_kv_gb300 import santa
from tests import kv4_util

DEV = "cuda"
OPS = ["kv4", "window"]
NINF = float("-inf")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def attend(op, q, k, v, seq, window=0, sinks=0, scale=0.0):
    """(the kernel's output, the definition's in 64 bits); q, k, v CPU bf16."""
    sl = torch.tensor(seq, dtype=torch.int32, device=DEV)
    if op == "kv4":
        parts = [torch.from_numpy(x) for t in (k, v) for x in kv4_util.quantise(t)]
        kr, vr = kv4_util.values(parts[0].numpy(), parts[1].numpy()), kv4_util.values(parts[2].numpy(), parts[3].numpy())
        out = santa.decode_kv4(q.to(DEV), santa.KV4Cache(*(x.to(DEV) for x in parts)), sl, window, sinks, scale)
    else:
        kr, vr = k.double().numpy(), v.double().numpy()
        out = santa.decode_window(q.to(DEV), k.to(DEV), v.to(DEV), sl, window, sinks, scale)
    return out.cpu().double().numpy(), kv4_util.attention(q, kr, vr, seq, window, sinks, scale)


# ------------------------------------------------------------------ very large scores

@pytest.mark.gpu
@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("d,H_kv,G", [(128, 2, 4), (128, 1, 8), (64, 2, 2), (64, 1, 8)])
@pytest.mark.parametrize("n", [48, 5008])
def test_scores_of_any_finite_size(op, d, H_kv, G, n):
    """Products of 1e3 to 1e37 of both signs: one key leads, or two do by exactly the same score,
    and the next is a step of the key's format behind.  Steps of at least 1/32 of a score of
    1e3 / sqrt(d): the others weigh less than 2^-5 there and nothing above; the weights are in
    the reference.  Tolerance: a weight is off by less than 1e-6 (exponent, its rounding), the
    output by twice that of max|v|."""
    g = gen(n + G)
    sizes = [1e3, 1e6, 3e7, 1e8, 2e8, 5e8, 1e9, 3e9, 1e12, 1e20, 1e30, 1e37]
    B = len(sizes)
    q = torch.zeros(B, H_kv * G, d)
    for b, s in enumerate(sizes):
        q[b, :, 5] = s * (1 + torch.rand(H_kv * G, generator=g))
    q[:, 1::2] *= -1
    q[:, :, 5] /= 6 * 2.0 ** 5
    k = torch.zeros(B, H_kv, n, d)
    grid = torch.tensor([0.5, 1, 1.5, 2, 3, 4])
    k[..., 5] = grid[torch.randint(0, 6, (B, H_kv, n), generator=g)] * 2.0 ** 5
    k[..., 5] *= torch.randint(0, 2, (B, H_kv, n), generator=g) * 2 - 1
    k[..., 6] = 6 * 2.0 ** 5                       # the group's largest: its scale is 2^5
    lead = torch.randint(0, n, (B, H_kv, 3), generator=g)
    for b in range(B):
        for h in range(H_kv):
            k[b, h, lead[b, h, 0], 5] = 6 * 2.0 ** 5
            k[b, h, lead[b, h, 1], 5] = -6 * 2.0 ** 5
            if b % 2:
                k[b, h, lead[b, h, 2], 5] = 6 * 2.0 ** 5
    v = torch.randn(B, H_kv, n, d, generator=g)
    got, want = attend(op, q.bfloat16(), k.bfloat16(), v.bfloat16(), [n - b % 3 for b in range(B)])
    assert np.abs(got - want).max() <= 2e-6 * float(v.abs().max())


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [0.0, 0.25, -0.1])
def test_a_score_of_minus_infinity_weighs_nothing(d, scale):
    """Keys that hold an infinity against a query of the other sign (so that the score is minus
    infinity), in visible places: single ones, whole tiles before any other key, and whole shares
    of other CTAs."""
    g = gen(d)
    n, B, H_kv, G = 6000, 3, 2, 4
    q = torch.randn(B, H_kv * G, d, generator=g)
    q[:, :, 3] = 1
    k, v = torch.randn(B, H_kv, n, d, generator=g) * 0.25, torch.randn(B, H_kv, n, d, generator=g)
    bad = float("inf") if scale < 0 else NINF
    k[0, :, torch.randint(0, n, (50,), generator=g), 3] = bad
    k[1, :, :2500, 3] = bad
    k[2, :, 100:, 3] = bad
    got, want = attend("window", q.bfloat16(), k.bfloat16(), v.bfloat16(), [n, n, n], scale=scale)
    assert np.abs(got - want).max() <= 1e-4 * float(v.abs().max())      # (scores are long sums here)


# ------------------------------------------------------------------ very small weights

@pytest.mark.gpu
@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("d,G", [(64, 4), (64, 8), (128, 4), (128, 8)])
@pytest.mark.parametrize("bits", [30, 33, 36])
@pytest.mark.parametrize("n,lead", [(32, 0), (32, 17), (32, 31), (3008, 0), (3008, 1500), (3008, 3007)])
def test_many_keys_of_very_small_weight(op, d, G, bits, n, lead):
    """One key leads and the others weigh less than 2^-bits of it (2^-37.1 at the least): v is 0 at
    the first and 6 at the others, so that the output is their share.  With the leading weight at
    2^9 theirs is 2^-28.1; held to 2^-35, half a step is 2^-7.9 of it."""
    q, k, v = torch.zeros(1, G, d), torch.zeros(1, 1, n, d), torch.full((1, 1, n, d), 6.0)
    q[:, :, 0] = 1.0
    k[..., 0] = -6.0
    k[0, 0, lead, 0] = 0
    v[0, 0, lead] = 0
    scale = bits * math.log(2) / 6 * 1.03
    got, want = attend(op, q.bfloat16(), k.bfloat16(), v.bfloat16(), [n], scale=scale)
    assert np.abs(got / want - 1).max() <= 2.0 ** -7


# ------------------------------------------------------------------ the terms of a weight

def two_keys(seed, d, H_kv, G, B=48, n=48):
    """Two keys that weigh 1 and w = exp(-q t), t and q of many sizes, at any two places of the
    sequence; the others nothing.  v is 0 and 6: the output is 6 w / (1 + w)."""
    g = gen(seed)
    q, k, v = torch.zeros(B, H_kv * G, d), torch.zeros(B, H_kv, n, d), torch.zeros(B, H_kv, n, d)
    q[:, :, 9] = 0.25 + torch.rand(B, H_kv * G, generator=g)
    k[..., 9] = -1024
    v[...] = torch.randn(B, H_kv, n, 1, generator=g)
    for b in range(B):
        for h in range(H_kv):
            i, j = torch.randperm(n, generator=g)[:2].tolist()
            k[b, h, i, 9], k[b, h, j, 9] = 0, -torch.rand(1, generator=g).item()
            v[b, h, i], v[b, h, j] = 0, 6
    return q.bfloat16(), k.bfloat16(), v.bfloat16()


# Error of 6 w / (1 + w).  w: its exponent is rounded near 2^3 (2^-21 ln 2), the factor log2 e by
# 2^-25 of at most 2.2, two exponentials are off by 2^-22 each: less than 9e-7, times 6 w / (1 + w)^2,
# at most 6 / 4.  The weight in two or three terms 2^-23, their sum and products in the tensor cores
# three steps of 2^-23, the sum of weights, the reciprocal and the product 2^-24, 2^-23 and 2^-24:
# six times 2^-23, times 6 w / (1 + w), at most 3.
TOL_TWO = 9e-7 * 1.5 + 6 * 2.0 ** -23 * 3


def many_keys(seed, d, H_kv, G, B=8, n=64):
    """Keys of comparable weight (scores within 4), v of both signs."""
    g = gen(seed)
    q, k = torch.zeros(B, H_kv * G, d), torch.zeros(B, H_kv, n, d)
    q[:, :, 9] = 0.25 + torch.rand(B, H_kv * G, generator=g)
    k[..., 9] = 3 * torch.rand(B, H_kv, n, generator=g)
    return q.bfloat16(), k.bfloat16(), torch.randn(B, H_kv, n, d, generator=g).bfloat16()


# Error of sum p v / sum p, relative to max|v|: twice that of a weight (9e-7); the tensor cores' sums,
# at most 6 steps of 2^-23 in a row, 64 / 16 additions of them and 8 of a lane's weights, 2^-24 each, and
# as much again as the exchange of both, the reciprocal and the product take.
TOL_MANY = 2 * 9e-7 + (12 + 4 + 8 + 6) * 2.0 ** -24


@pytest.mark.gpu
@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_a_weight_keeps_its_bits(op, d, G):
    q, k, v = two_keys(d + G, d, 2, G)
    got, want = attend(op, q, k, v, [48] * 48, scale=1.0)
    assert np.abs(got - want).max() <= TOL_TWO
    q, k, v = many_keys(d + G, d, 2, G)
    got, want = attend(op, q, k, v, [64] * 8, scale=1.0)
    assert np.abs(got - want).max() <= TOL_MANY * float(v.abs().max())


def error_with(terms, op, q, k, v):
    """Largest error of the output in 64 bits when each weight is the sum of its first `terms` terms."""
    if op == "kv4":
        k, v = (torch.from_numpy(kv4_util.values(*kv4_util.quantise(x))) for x in (k, v))
    s = torch.einsum("bhgd,bhnd->bhgn", q.double().view(k.shape[0], k.shape[1], -1, q.shape[-1]), k.double())
    p = torch.exp(s - s.amax(-1, keepdim=True)) * 512
    kept = torch.zeros_like(p)
    for _ in range(terms):
        kept += (p - kept).to(torch.float16 if op == "kv4" else torch.bfloat16).double()
    return float(torch.einsum("bhgn,bhnd->bhgd", (p - kept) / p.sum(-1, keepdim=True), v.double()).abs().max())


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_the_tolerances_would_show_a_lost_term(op, d, G):
    """The same inputs with the last term of each weight left out (many keys: all but the first):
    beyond twice the tolerance."""
    q, k, v = two_keys(d + G, d, 2, G)
    assert error_with(1 if op == "kv4" else 2, op, q, k, v) > 2 * TOL_TWO
    q, k, v = many_keys(d + G, d, 2, G)
    assert error_with(1, op, q, k, v) > 2 * TOL_MANY * float(v.abs().max())
