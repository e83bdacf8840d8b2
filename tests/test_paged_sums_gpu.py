"""The size of the errors of attention over a paged cache, against 64 bits: sums of up to 524288 values of one
sign, which a one-sided rounding on the way would move all alike, and the root mean square of the error."""
import math

import pytest
import torch

from stochastic_sparse_kv_gb300 import santa

pytestmark = pytest.mark.gpu
DEV = "cuda"
bf16 = torch.bfloat16
PAGE, PAGES = 256, 64   # a pool of few pages, which stand in the tables many times


def cache_of(B, H_kv, d, n, seed, q_scale):
    g = torch.Generator(device=DEV).manual_seed(seed)
    v = (1.0 + 0.6 * torch.rand(PAGES, H_kv, PAGE, d, generator=g, device=DEV)).to(bf16)
    k = (q_scale * torch.randn(PAGES, H_kv, PAGE, d, generator=g, device=DEV)).to(bf16)
    table = torch.randint(0, PAGES, (B, n // PAGE), generator=g, device=DEV, dtype=torch.int32)
    return santa.PagedCache(k, v, table)


# B * H_kv above the number of SMs: shares hold all the keys of an item.  The tensor cores cut off instead of
# rounding: for every 16 keys each product below 2^-25 of the power of 2 in the sum, and the new sum below 2^-23 of
# it (test_what_the_tensor_cores_keep), together 16 2^-25 + 2^-23 = 5 2^-23 of the sum at the most, half of that on
# average.  They add up 256 tiles of 128 keys at a time, 2048 steps of a sum that grows from 0: 2048 / 2 of these, 5 2^-13,
# on average half of it.  The rest is rounded to the nearest.
CUT = 5 * 2.0 ** -13


@pytest.mark.parametrize("together,kept", [(1, 23), (2, 24), (4, 25), (16, 25)])
@pytest.mark.parametrize("first", [1024.0, -1024.0])
def test_what_the_tensor_cores_keep(together, kept, first):
    """Weights of 1, a value of 2^10, then in six steps `together` values 2^-j of it each, then its negative: what is left
    is what the sums kept.  (If this changes, so do the bounds below.)"""
    n, d, page = 128, 64, 16
    j = 17 + torch.arange(d, dtype=torch.float64) % 16
    v = torch.zeros(n, d, dtype=torch.float64)
    v[64], v[48] = first, -first    # (the upper half of a tile comes first)
    for step in (80, 96, 112, 0, 16, 32):
        v[step:step + together] = abs(first) * 2.0 ** -j
    pool = v.to(bf16).view(n // page, 1, page, d).to(DEV)
    table = torch.arange(n // page, dtype=torch.int32, device=DEV)[None]
    out = santa.attend_paged(torch.zeros(1, 1, 1, d, dtype=bf16, device=DEV), santa.PagedCache(torch.zeros_like(pool), pool, table),
                             torch.tensor([n - 1], dtype=torch.int32, device=DEV))[0, 0, 0].double().cpu() * n
    if first > 0:   # (where it is negative, what is cut off is the other way round)
        assert torch.equal(out, torch.where(j <= kept, 6 * together * abs(first) * 2.0 ** -j, 0.0).to(bf16).double())
    else:
        assert torch.equal(out[j <= kept - 1], (6 * together * abs(first) * 2.0 ** -j).to(bf16).double()[j <= kept - 1])


@pytest.mark.parametrize("T,d,G,n", [(1, 128, 4, 524288), (1, 64, 8, 524288), (1, 128, 4, 40960), (1, 64, 4, 131072), (40, 128, 4, 131072),
                                     (70, 64, 2, 131072), (33, 128, 8, 33280), (5, 128, 2, 65536 + 512)])
def test_long_sums_of_one_sign(T, d, G, n):
    """Scores all 0: the mean of the values."""
    B, H_kv = 40, 4 if T > 1 else 8
    cache = cache_of(B, H_kv, d, n, n + T, 1.0)
    q = torch.zeros(B, T, H_kv * G, d, dtype=bf16, device=DEV)
    got = santa.attend_paged(q, cache, torch.full((B,), n - T, dtype=torch.int32, device=DEV))[:, -1].double()
    page_sums = cache.v.double().sum(2)
    ref = torch.stack([page_sums[cache.table[b].long()].sum(0) for b in range(B)]) / n
    ref = ref.repeat_interleave(G, 1)
    assert ((got - ref).abs() <= (2.0 ** -8 + CUT) * ref).all()
    rounded = ref.to(bf16).double()
    bias = float(((got - rounded) / ref).mean())
    # (rounding moves the mean by what the results are moved, and of 10^5 by chance by a thousandth of a step)
    assert abs(bias) <= CUT / 2 + 2.0 ** -18, bias


@pytest.mark.parametrize("T,d,n,window", [(1, 128, 300032, 0), (1, 64, 131072, 0), (34, 128, 131072, 0), (3, 64, 262144, 100000)])
def test_long_sums_of_weights(T, d, n, window):
    """Scores of every size: the last token of a few heads against 64 bits."""
    B, H_kv, G = 40, 4, 4
    cache = cache_of(B, H_kv, d, n, n, 1.0)
    g = torch.Generator(device=DEV).manual_seed(d)
    q = (0.7 * torch.randn(B, T, H_kv * G, d, generator=g, device=DEV)).to(bf16)
    got = santa.attend_paged(q, cache, torch.full((B,), n - T, dtype=torch.int32, device=DEV), window=window, sinks=5)[:, -1].double()
    err, bias = [], []
    for b, h in ((0, 0), (B - 1, H_kv - 1), (17, 2)):
        rows = cache.table[b].long()
        k, v = (x[rows, h].reshape(-1, d)[:n].double() for x in cache[:2])
        s = q[b, -1, h * G:(h + 1) * G].double() @ k.T / math.sqrt(d)
        if window:
            s[:, 5:n - window] = -math.inf
        p = torch.softmax(s, -1)
        ref = p @ v
        err.append((got[b, h * G:(h + 1) * G] - ref) / ref)
        bias.append((got[b, h * G:(h + 1) * G] - ref.to(bf16).double()) / ref)
        # the weights' own rounding: by 2^-8 of a weight times the value's distance from the result, of 0.35 at most; of
        # thousands of keys with weights like these a hundredth of that is left (the root of the sum of p^2 is below 1/30)
        assert float(p.pow(2).sum(-1).max()) <= 1 / 900
        assert (err[-1].abs() <= 2.0 ** -8 + CUT + 2.0 ** -8 * 0.35 * 4 / 30).all()
    # A cut of all alike is in the mean, beside what the same rounding does to the results that it should give (they lie
    # close together on the grid of bf16, so that is not 0).  By chance: weights move a result by 2^-8 / sqrt(12) of 0.18
    # (the values' deviation) / 30, 7e-6, and its rounding with 7e-6 / 2^-7.4 = 0.0012 of them, by a step of 2^-7.4 each:
    # the mean of 768 by 2^-7.4 sqrt(0.0012 / 768) = 7e-6, here four times
    assert abs(float(torch.stack(bias).mean())) <= CUT / 2 + 2.0 ** -15


@pytest.mark.parametrize("T,d,G", [(1, 128, 4), (1, 64, 8), (40, 128, 4), (200, 64, 1)])
@pytest.mark.parametrize("rise", [-25, 25, 60])
def test_scores_that_rise_or_fall_from_chain_to_chain(T, d, G, rise):
    """Keys of weight 1 and then of 2^rise, 32768 each and some; the values of those that weigh less are larger by as
    much, so that both halves count alike."""
    B, H_kv, n = 40, 8 if T == 1 else 4, 66048
    half = n // 2 // PAGE
    k = torch.zeros(2, H_kv, PAGE, d, dtype=bf16, device=DEV)
    k[1, ..., 0] = rise
    v = torch.empty(2, H_kv, PAGE, d, dtype=bf16, device=DEV)
    small, large = (0, 1) if rise > 0 else (1, 0)
    v[small], v[large] = 2.0 ** abs(rise), 1.5
    table = torch.zeros(B, n // PAGE, dtype=torch.int32, device=DEV)
    table[:, half:] = 1
    q = torch.zeros(B, T, H_kv * G, d, dtype=bf16, device=DEV)
    q[..., 0] = 1.0
    got = santa.attend_paged(q, santa.PagedCache(k, v, table), torch.full((B,), n - T, dtype=torch.int32, device=DEV), scale=math.log(2.0))
    for t in {0, T // 2, T - 1}:
        a, b = half * PAGE, n - T + 1 + t - half * PAGE   # keys of either half that token t sees
        w = 2.0 ** rise
        want = (a * float(v[0, 0, 0, 0]) + w * b * float(v[1, 0, 0, 0])) / (a + w * b)
        # (the scale is rounded to 2^-25 of it: a weight of 2^60 by 60 2^-25)
        assert float((got[:, t].double() / want - 1).abs().max()) <= 2.0 ** -8 + CUT + 2.0 ** -18


@pytest.mark.parametrize("B,T,H_kv,G,d,n,window", [(8, 1, 4, 4, 128, 4096, 0), (2, 1, 4, 8, 64, 20000, 0), (4, 5, 2, 4, 128, 9000, 4096),
                                                   (2, 300, 2, 4, 128, 5000, 0), (2, 130, 2, 8, 64, 1500, 600), (1, 64, 8, 1, 128, 400, 0)])
@pytest.mark.parametrize("std", [0.5, 3.0])
def test_root_mean_square_error(B, T, H_kv, G, d, n, window, std):
    """Values of both signs: the result's rounding, and one rounding of each weight, e_j, in the sums of weights and of
    values alike: sum p_j e_j (v_j - o).  The relative error of a bf16 rounding has the root mean square 2^-7 / sqrt(12) of
    the number's power of 2, and E[2^-2x] = 0.541 of mantissas 2^x whose logarithms are even; errors of keys are independent."""
    g = torch.Generator(device=DEV).manual_seed(n + d)
    cols = -(-n // 64)
    k, v = (torch.randn(B * cols, H_kv, 64, d, generator=g, device=DEV).to(bf16) for _ in range(2))
    table = torch.arange(B * cols, device=DEV, dtype=torch.int32).view(B, cols)
    x = torch.randn(B, T, H_kv * G, d, generator=g, device=DEV)
    q = (std * math.sqrt(d) * x / x.norm(dim=-1, keepdim=True)).to(bf16)
    got = santa.attend_paged(q, santa.PagedCache(k, v, table), torch.full((B,), n - T, dtype=torch.int32, device=DEV), window=window)
    u = 2.0 ** -7 * math.sqrt(0.541 / 12)
    error, expected, size, count = 0.0, 0.0, 0.0, 0
    for b in range(B):
        for t in sorted({0, T // 2, T - 1}):
            P = n - T + t
            lo = max(0, P - window + 1) if window else 0
            kb, vb = (x[table[b].long()].transpose(1, 2).flatten(0, 1)[lo:P + 1].double() for x in (k, v))   # [keys, H_kv, d]
            s = torch.einsum("hgd,nhd->hgn", q[b, t].double().view(H_kv, G, d), kb) / math.sqrt(d)
            p = torch.softmax(s, -1)
            o = torch.einsum("hgn,nhd->hgd", p, vb)
            moved = torch.einsum("hgn,nhd->hgd", p.pow(2), vb.pow(2)) - 2 * o * torch.einsum("hgn,nhd->hgd", p.pow(2), vb) + \
                o.pow(2) * p.pow(2).sum(-1, keepdim=True)
            error += float((got[b, t].double().view_as(o) - o).pow(2).sum())
            expected += float((o.to(bf16).double() - o).pow(2).sum() + u * u * moved.sum())
            size += float(o.pow(2).sum())
            count += o.numel()
    print("rms", math.sqrt(error / size), "of", math.sqrt(expected / size))
    # (thousands of results: chance leaves a few hundredths)
    assert count >= 2000 and error <= 1.1 ** 2 * expected
