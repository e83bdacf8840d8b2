"""Attention over a paged cache with values that are not finite: at keys that weigh nothing, many of them with
two row tiles at once, and the same bits at every call."""
import math

import pytest
import torch

from stochastic_sparse_kv_gb300 import santa

pytestmark = pytest.mark.gpu
DEV = "cuda"
bf16 = torch.bfloat16


def problem(B, T, H_kv, G, d, page, n, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    cols = -(-n // page)
    k, v = (torch.randn(B * cols, H_kv, page, d, generator=g, device=DEV).to(bf16) for _ in range(2))
    table = torch.randperm(B * cols, generator=g, device=DEV).view(B, cols).to(torch.int32)
    q = torch.randn(B, T, H_kv * G, d, generator=g, device=DEV).to(bf16)
    return q, santa.PagedCache(k, v, table), torch.full((B,), n - T, dtype=torch.int32, device=DEV)


def put(pool, table, b, h, j, c, x):
    page = pool.shape[2]
    pool[int(table[b, j // page]), h, j % page, c] = x


@pytest.mark.parametrize("T,n,H_kv,B", [(1, 500, 2, 1), (1, 40000, 2, 1), (20, 3000, 2, 2), (300, 1000, 2, 1), (300, 9000, 8, 2)])
@pytest.mark.parametrize("d,G", [(64, 4), (128, 2), (128, 8)])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("window,sinks", [(0, 0), (260, 3)])
def test_a_value_that_is_not_finite_at_a_key_of_no_weight(T, n, H_kv, B, d, G, value, window, sinks):
    """A score of minus infinity and a value that is not finite at one key, where all tokens see it and where
    some do: that feature of those that see it is not finite (an infinity or NaN), all else is what it is with
    a zero there, bit for bit."""
    q, cache, pos = problem(B, T, H_kv, G, d, 16, n, T + d)
    q[..., 3] = 1.0
    # all see the first two (with a window: none; the sink and a key of the last window do), the chunk's keys some
    keys = [(2, 1), (200, 5), (n - T - 20, 7), (n - T, 8), (n - 1 - T // 2, 9), (n - 1, d - 1)]
    for j, c in keys:
        put(cache.k, cache.table, 0, 0, j, 3, -math.inf)
        put(cache.v, cache.table, 0, 0, j, c, 0.0)
    want = santa.attend_paged(q, cache, pos, window=window, sinks=sinks)
    assert torch.isfinite(want).all()
    for j, c in keys:
        put(cache.v, cache.table, 0, 0, j, c, value)
    got = santa.attend_paged(q, cache, pos, window=window, sinks=sinks)
    hit = torch.zeros_like(want, dtype=torch.bool)
    P = torch.arange(n - T, n, device=DEV)
    for j, c in keys:
        sees = j <= P
        if window:
            sees &= (j > P - window) | torch.tensor(j < sinks, device=DEV)
        hit[0, :, :G, c] |= sees[:, None]
    assert hit.any()
    assert not torch.isfinite(got[hit]).any()
    assert torch.equal(got[~hit], want[~hit])


@pytest.mark.parametrize("d,G", [(64, 8), (128, 4), (128, 1)])
@pytest.mark.parametrize("window", [0, 150])
def test_many_values_that_are_not_finite_the_same_bits_every_time(d, G, window):
    """Two row tiles find and clear the same values at the same time; each token has those it sees."""
    T, n = 700, 1100
    q, cache, pos = problem(2, T, 2, G, d, 64, n, d + G)
    plain = santa.attend_paged(q, cache, pos, window=window)
    g = torch.Generator().manual_seed(1)
    hit = torch.zeros_like(plain, dtype=torch.bool)
    P = torch.arange(n - T, n, device=DEV)
    for _ in range(60):
        b, h, j, c = (int(torch.randint(0, m, (1,), generator=g)) for m in (2, 2, n, d))
        put(cache.v, cache.table, b, h, j, c, (math.inf, -math.inf, math.nan)[int(torch.randint(0, 3, (1,), generator=g))])
        sees = (j <= P) & ((j > P - window) if window else True)
        hit[b, :, h * G:(h + 1) * G, c] |= sees[:, None]
    first = None
    for _ in range(40):
        got = santa.attend_paged(q, cache, pos, window=window)
        bits = got.view(torch.int16)
        first = bits if first is None else first
        assert torch.equal(bits, first)
    assert not torch.isfinite(got[hit]).any() and torch.isfinite(got[~hit]).all()
    # (a value of a feature is a zero in its place for the others: the bits of features without any are as before)
    clean = ~hit.any(1, keepdim=True).expand_as(hit)
    assert torch.equal(got[clean], plain[clean])
