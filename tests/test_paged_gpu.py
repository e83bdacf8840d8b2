"""Rotary positions, writing into a paged cache and attention over it on the GPU, against their
formulas in 64 bits (tests/paged_util.py)."""
import ctypes
import itertools
import math

import numpy as np
import pytest
import torch

from stochastic_sparse_kv_gb300 import santa
from tests import paged_util as pu

pytestmark = pytest.mark.gpu
DEV = "cuda"
bf16 = torch.bfloat16


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rand(g, *shape):
    return torch.randn(*shape, generator=g).to(bf16)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def f64(t):
    return t.detach().cpu().double().numpy()


# ------------------------------------------------------------------ rope

def check_rope(got, x, f, amplitude, layout, pos, counts, before):
    """Rotated where live, as before elsewhere.  Half a step of bf16, and of fp32 the angle's
    rounding (2^-24 pi), two products and their sum, times both features."""
    ref = pu.rotate(x, f, amplitude, layout, pos)
    size = np.abs(f64(x)).max(-1, keepdims=True) * amplitude
    rot = 2 * len(f)
    for b, n in enumerate(counts):
        g = f64(got)[b, :n]
        r = ref[b, :n]
        assert (np.abs(g - r) <= 2.0 ** -8 * np.abs(r) + 2.0 ** -20 * size[b, :n]).all()
        assert np.array_equal(g[..., rot:], f64(x)[b, :n, :, rot:])
        assert torch.equal(got[b, n:], before[b, n:])


@pytest.mark.parametrize("layout", ["halves", "pairs"])
@pytest.mark.parametrize("d,rot", [(64, 16), (64, 48), (64, 64), (128, 16), (128, 80), (128, 128)])
@pytest.mark.parametrize("B,T,H", [(1, 1, 1), (3, 21, 5), (2, 130, 8)])
def test_rope(layout, d, rot, B, T, H):
    g = gen(d + rot + T)
    t = santa.rope_table(rot, 500000.0, layout, "ramp", 4.0, original=4096)
    f, amplitude = pu.frequencies(rot, 500000.0, "ramp", 4.0, original=4096)
    x = rand(g, B, T, H, d)
    pos = [int(v) for v in torch.randint(0, 5000, (B,), generator=g)]
    pos[-1] = 0
    got = santa.rope(x.to(DEV), t, ints(pos))
    check_rope(got, x, f, amplitude, layout, pos, [T] * B, got)
    # padded rows, rows given, in place
    counts = [T, 0, T // 2][:B]
    out = torch.full((B, T, H, d), 7.0, dtype=bf16, device=DEV)
    before = out.clone()
    assert santa.rope(x.to(DEV), t, ints(pos), ints(counts), out=out) is out
    check_rope(out, x, f, amplitude, layout, pos, counts, before)
    y = x.to(DEV)
    santa.rope(y, t, ints(pos), ints(counts), out=y)
    check_rope(y, x, f, amplitude, layout, pos, counts, x.to(DEV))
    fresh = santa.rope(x.to(DEV), t, ints(pos), ints(counts))
    check_rope(fresh, x, f, amplitude, layout, pos, counts, torch.zeros_like(fresh))


@pytest.mark.parametrize("layout", ["halves", "pairs"])
def test_rope_far_positions_and_fast_angles(layout):
    """Positions up to the largest there is: the fastest pair turns a radian a position."""
    g = gen(5)
    x = rand(g, 6, 2, 3, 128)
    pos = [131071, 524286, 1 << 20, (1 << 24) + 1, (1 << 30) + 12345, (1 << 31) - 3]
    t = santa.rope_table(128, layout=layout)
    f, _ = pu.frequencies(128)
    # the reference's own product p f is off by 2^-53 of the angle: 2^-22 at 2^31
    got = santa.rope(x.to(DEV), t, ints(pos))
    check_rope(got, x, f, 1.0, layout, pos, [2] * 6, got)


def test_rope_small_angles_keep_their_bits():
    """x = 0, y = 1: the result is -sin of angles down to 1e-6, each to half a step."""
    f, _ = pu.frequencies(128, 1e6)
    t = santa.rope_table(128, 1e6)
    x = torch.zeros(1, 4, 1, 128, dtype=bf16)
    x[..., 64:] = 1
    got = f64(santa.rope(x.to(DEV), t, ints([1])))
    ref = pu.rotate(x, f, 1.0, "halves", [1])
    assert (np.abs(got - ref) <= (2.0 ** -8 + 2.0 ** -20) * np.abs(ref)).all()


@pytest.mark.parametrize("d", [64, 128])
def test_rope_strides(d):
    """Slices of one projection, heads outermost, one row for the whole batch; into strided rows."""
    g = gen(d)
    B, T, H = 3, 19, 4
    t = santa.rope_table(d, layout="pairs")
    f, _ = pu.frequencies(d)
    fused = rand(g, B, T, 3 * H, d).to(DEV)
    for x in (fused[:, :, H:2 * H], rand(g, B, H, T, d).to(DEV).transpose(1, 2), rand(g, 1, T, H, d).to(DEV).expand(B, T, H, d),
              rand(g, B, T, 1, d).to(DEV).expand(B, T, H, d)):
        room = torch.full((B, H, T, d + 8), 3.0, dtype=bf16, device=DEV)
        out = room.transpose(1, 2)[..., :d]
        santa.rope(x, t, ints([4, 0, 100]), out=out)
        check_rope(out, x.cpu(), f, 1.0, "pairs", [4, 0, 100], [T] * B, out)
        assert (room[..., d:] == 3).all()
    # in place in the projection: nothing else changes
    kept = fused.clone()
    part = fused[:, :, H:2 * H]
    santa.rope(part, t, ints([4, 0, 100]), out=part)
    check_rope(part, kept[:, :, H:2 * H].cpu(), f, 1.0, "pairs", [4, 0, 100], [T] * B, part)
    assert torch.equal(fused[:, :, :H], kept[:, :, :H]) and torch.equal(fused[:, :, 2 * H:], kept[:, :, 2 * H:])


def test_rope_skips_rows_out_of_range():
    g = gen(9)
    x = rand(g, 6, 3, 2, 64).to(DEV)
    t = santa.rope_table(64)
    ws = santa.new_workspace(65536, DEV)
    out = torch.full_like(x, 5.0)
    santa.rope(x, t, ints([0, -1, 5, 7, (1 << 31) - 1, (1 << 31) - 2]), ints([3, 1, 4, -1, 1, 1]), out=out, workspace=ws)
    assert santa.device_status(ws) == santa.DEV_BAD_POSITION
    assert (out[1:5] == 5).all() and (out[0] != 5).any() and (out[5, 0] != 5).any() and (out[5, 1:] == 5).all()
    assert santa.device_status(ws) == 0


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("d,layout", [(64, "pairs"), (128, "halves")])
@pytest.mark.parametrize("with_q", [False, True])
def test_append(page, d, layout, with_q):
    """Rows that begin and end inside pages, rotated, with and without queries; all else stays."""
    g = gen(page + d)
    B, T, H_q, H_kv = 4, 37, 8, 2
    pos, counts = [page - 1, 0, 3 * page - 37, 2 * page], [37, 0, 37, 1]
    cols = -(-(max(pos) + T) // page)
    table, n_pages = pu.pages(g, [p + c for p, c in zip(pos, counts)], page, cols)
    qkv = rand(g, B, T, H_q + 2 * H_kv, d).to(DEV)
    q, k, v = qkv.split((H_q, H_kv, H_kv), 2)
    t = santa.rope_table(d // 2, layout=layout)
    f, _ = pu.frequencies(d // 2)
    pools = [torch.full((n_pages, H_kv, page, d), 9.0, dtype=bf16, device=DEV) for _ in range(2)]
    cache = santa.PagedCache(*pools, table.to(DEV))
    q_out = torch.full((B, T, H_q, d), 5.0, dtype=bf16, device=DEV)
    ws = santa.new_workspace(65536, DEV)
    got = santa.paged_append(cache, k, v, ints(pos), ints(counts), rope=t, q=q if with_q else None,
                             q_out=q_out if with_q else None, workspace=ws)
    assert santa.device_status(ws) == 0
    assert got is (q_out if with_q else None)
    if with_q:
        check_rope(q_out, q.cpu(), f, 1.0, layout, pos, counts, torch.full_like(q_out, 5.0))
    want = pu.rotate(k.cpu(), f, 1.0, layout, pos)
    held_k, held_v = f64(pools[0]), f64(pools[1])
    seen = np.zeros(held_k.shape, dtype=bool)
    for b in range(B):
        for i in range(counts[b]):
            p, r = int(table[b, (pos[b] + i) // page]), (pos[b] + i) % page
            assert (np.abs(held_k[p, :, r] - want[b, i]) <= 2.0 ** -8 * np.abs(want[b, i]) + 2.0 ** -18).all()
            assert np.array_equal(held_v[p, :, r], f64(v[b, i]))
            seen[p, :, r] = True
    assert (held_k[~seen] == 9).all() and (held_v[~seen] == 9).all()
    # without a rotation: the rows themselves
    santa.paged_append(cache, k, v, ints(pos), ints(counts))
    for b in range(B):
        for i in range(counts[b]):
            p, r = int(table[b, (pos[b] + i) // page]), (pos[b] + i) % page
            assert torch.equal(pools[0][p, :, r], k[b, i]) and torch.equal(pools[1][p, :, r], v[b, i])


def test_append_skips_what_has_no_place():
    """Positions out of range skip the row, tokens without a page are left out alone."""
    g = gen(3)
    B, T, H, d, page = 5, 20, 2, 64, 16
    k, v, q = (rand(g, B, T, h, d).to(DEV) for h in (H, H, 4))
    table = ints([[0, 1, 2], [3, -1, 4], [5, 8, 6], [7, 0, 0], [0, 0, 0]])
    cache = santa.PagedCache(*(torch.full((8, H, page, d), 9.0, dtype=bf16, device=DEV) for _ in range(2)), table)
    ws = santa.new_workspace(65536, DEV)
    q_out = torch.full_like(q, 5.0)
    pos = [0, 10, 14, -1, 40]
    santa.paged_append(cache, k, v, ints(pos), rope=santa.rope_table(64), q=q, q_out=q_out, workspace=ws)
    assert santa.device_status(ws) == santa.DEV_BAD_POSITION | santa.DEV_BAD_PAGE
    f, _ = pu.frequencies(64)
    check_rope(q_out, q.cpu(), f, 1.0, "halves", [0, 10, 14, 0, 0], [T, T, T, 0, 0], torch.full_like(q, 5.0))
    for pool, new in ((cache.v, v),):
        assert torch.equal(pool[0], new[0, :16].transpose(0, 1)) and torch.equal(pool[1][:, :4], new[0, 16:].transpose(0, 1))
        assert torch.equal(pool[3][:, 10:], new[1, :6].transpose(0, 1)) and (pool[3][:, :10] == 9).all() and (pool[4] == 9).all()
        assert torch.equal(pool[5][:, 14:], new[2, :2].transpose(0, 1)) and torch.equal(pool[6][:, :2], new[2, 18:].transpose(0, 1))
        assert (pool[2] == 9).all() and (pool[7] == 9).all()


@pytest.mark.parametrize("d", [64, 128])
def test_append_as_many_tokens_as_there_may_be(d):
    """2^31 - 1 groups of features, or the most below, of which few tokens are live (one row stands for
    them all: token stride 0)."""
    T = ((1 << 31) - 1) // (2 * (d // 16))
    row = rand(gen(d), 1, 1, 1, d).to(DEV)
    cache = santa.PagedCache(*(torch.zeros(4, 1, 16, d, dtype=bf16, device=DEV) for _ in range(2)), ints([[2, 0, 3]]))
    santa.paged_append(cache, row.expand(1, T, 1, d), row.expand(1, T, 1, d), ints([14]), ints([3]))
    for pool in (cache.k, cache.v):
        assert torch.equal(pool[2, 0, 14:], row[0, 0].expand(2, d)) and torch.equal(pool[0, 0, 0], row[0, 0, 0])
        assert not pool[2, 0, :14].any() and not pool[0, 0, 1:].any() and not pool[1].any() and not pool[3].any()
    with pytest.raises(santa.SantaError):
        santa.paged_append(cache, row.expand(1, T + 1, 1, d), row.expand(1, T + 1, 1, d), ints([14]), ints([3]))


# ------------------------------------------------------------------ attend

def problem(g, B, T, H_kv, G, d, page, lengths, counts, std=3.0, extra=0):
    """(q, k pool, v pool, table, pos) on the CPU; lengths with the chunk.  What no key holds is NaN."""
    pos = [n - c for n, c in zip(lengths, counts)]
    cols = -(-max(lengths + [T]) // page) + extra
    table, n_pages = pu.pages(g, lengths, page, cols)
    x = torch.randn(B, T, H_kv * G, d, generator=g)
    q = (std * math.sqrt(d) * x / x.norm(dim=-1, keepdim=True)).to(bf16)
    pools = []
    for _ in range(2):
        pool = torch.full((n_pages, H_kv, page, d), math.nan, dtype=bf16)
        for b, n in enumerate(lengths):
            for i in range(-(-n // page)):
                m = min(page, n - i * page)
                pool[int(table[b, i]), :, :m] = rand(g, H_kv, m, d)
        pools.append(pool)
    return q, *pools, table, pos


def check(got, want, spread, counts, before=None):
    got = f64(got)
    for b, n in enumerate(counts):
        g, w = got[b, :n], want[b, :n]
        assert np.array_equal(np.isnan(g), np.isnan(w)), f"row {b}: NaN in other places"
        fine = np.isfinite(w)
        assert np.array_equal(g[~fine & ~np.isnan(w)], w[~fine & ~np.isnan(w)])
        err = np.abs(g[fine] - w[fine])
        tol = pu.tolerance(w[fine], spread[b, :n][fine])
        assert (err <= tol).all(), f"row {b}: {(err - tol).max()} beyond, {(err / np.maximum(tol, 1e-30)).max()} of it"
        if before is not None:
            assert torch.equal(before[b, n:].cpu(), torch.from_numpy(got[b, n:]).to(bf16))


def attend(q, k, v, table, pos, counts=None, window=0, sinks=0, scale=0.0, **kw):
    cache = santa.PagedCache(k.to(DEV), v.to(DEV), table.to(DEV))
    return santa.attend_paged(q.to(DEV), cache, ints(pos), ints(counts) if counts is not None else None, window, sinks, scale, **kw)


SHAPES = [  # T, lengths: one token, a few, odd ones, more than a tile of rows, all of a sequence
    (1, [1, 2, 127]), (1, [128, 129, 1000]), (2, [2, 65, 300]), (5, [5, 133, 128]), (16, [16, 40, 640]), (33, [33, 129, 200]),
    (64, [64, 128, 777]), (65, [65, 400, 66]), (129, [129, 300, 131]), (257, [257, 700, 258]),
]


@pytest.mark.parametrize("T,lengths", SHAPES)
@pytest.mark.parametrize("d,G,H_kv,page", [(128, 4, 2, 64), (64, 8, 1, 16), (128, 1, 2, 128), (64, 2, 2, 256), (128, 8, 1, 32),
                                           (64, 1, 1, 64), (64, 4, 2, 128), (128, 2, 1, 16)])
def test_attend(T, lengths, d, G, H_kv, page):
    g = gen(T + d + G)
    p = problem(g, 3, T, H_kv, G, d, page, lengths, [T] * 3)
    want, spread = pu.attention(*p)
    check(attend(*p), want, spread, [T] * 3)


@pytest.mark.parametrize("d,G,page", [(128, 4, 16), (64, 8, 64), (128, 1, 128)])
@pytest.mark.parametrize("T,lengths,counts", [(40, [40, 300, 0, 513, 77], [40, 17, 0, 1, 39]), (150, [150, 150, 1, 600, 149], [150, 1, 0, 149, 75]),
                                              (3, [1, 0, 259, 31, 3], [1, 0, 3, 2, 0])])
def test_attend_ragged(d, G, page, T, lengths, counts):
    """Padded chunks, finished rows (no live token) and empty ones; rows past a count stay."""
    g = gen(T + G)
    p = problem(g, 5, T, 2, G, d, page, lengths, counts)
    want, spread = pu.attention(*p, counts)
    out = torch.full((5, T, 2 * G, d), 7.0, dtype=bf16, device=DEV)
    before = out.clone()
    assert attend(*p, counts, out=out) is out
    check(out, want, spread, counts, before)
    check(attend(*p, counts), want, spread, counts, torch.zeros_like(out))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (64, 4), (100, 0), (128, 130), (129, 16), (500, 400), (10000, 3), (200, 1000)])
@pytest.mark.parametrize("d,G,page,T,lengths", [(128, 4, 64, 1, [1, 450, 800]), (64, 8, 16, 37, [37, 333, 900]),
                                                (128, 2, 128, 260, [260, 511, 1023]), (64, 1, 32, 300, [300, 640, 900])])
def test_attend_window(window, sinks, d, G, page, T, lengths):
    g = gen(window + T)
    p = problem(g, 3, T, 1, G, d, page, lengths, [T] * 3)
    want, spread = pu.attention(*p, None, window, sinks)
    check(attend(*p, None, window, sinks), want, spread, [T] * 3)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("d,G,T", [(128, 4, 70), (64, 2, 140), (128, 1, 300), (64, 8, 3)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 2)])
def test_values_that_a_token_does_not_see_do_not_reach_it(bad, d, G, T, window, sinks):
    """Infinities and NaN in V at single features of keys inside the chunk, at the window's edge and
    before it: tokens that see the key have them at that feature, the others are as without."""
    g = gen(T)
    n = T + 170
    q, k, v, table, pos = problem(g, 2, T, 2, G, d, 16, [n, n - 5], [T, T])
    for b, h, j, c in ((0, 0, n - T + T // 2, 3), (0, 1, n - 1, d - 1), (1, 0, n - T + 4, 17), (1, 1, 60, 40), (1, 1, 1, 0)):
        v[int(table[b, j // 16]), h, j % 16, c] = bad
    want, spread = pu.attention(q, k, v, table, pos, None, window, sinks)
    assert np.isfinite(want).any() and not np.isfinite(want).all()
    check(attend(q, k, v, table, pos, None, window, sinks), want, spread, [T, T])


@pytest.mark.parametrize("d,G,T", [(128, 4, 70), (64, 1, 300), (64, 8, 3)])
def test_keys_that_a_token_does_not_see_do_not_reach_it(d, G, T):
    """The same in K: a NaN key makes those that see it NaN, wholly, and no others."""
    g = gen(T)
    n = T + 170
    q, k, v, table, pos = problem(g, 2, T, 2, G, d, 16, [n, n - 5], [T, T])
    for b, h, j, c in ((0, 0, n - T + T // 2, 3), (0, 1, n - 1, d - 1), (1, 0, n - 6, 17)):
        k[int(table[b, j // 16]), h, j % 16, c] = math.nan
    want, spread = pu.attention(q, k, v, table, pos)
    assert np.isfinite(want).any() and not np.isfinite(want).all()
    check(attend(q, k, v, table, pos), want, spread, [T, T])


@pytest.mark.parametrize("d,T", [(128, 1), (128, 90), (64, 4), (64, 200)])
def test_scores_of_minus_infinity_weigh_nothing(d, T):
    """Keys that hold an infinity against a query of the other sign: single ones, whole tiles before
    any other key, all that a token sees (then its result is NaN)."""
    g = gen(d + T)
    B, G, n = 3, 4, T + 700
    q, k, v, table, pos = problem(g, B, T, 1, G, d, 64, [n] * B, [T] * B, std=1.0)
    q[..., 3] = 1.0
    for b, keys in ((0, [5, 130, 131, 300, n - T - 1]), (1, range(400)), (2, range(n - T + 1))):
        for j in keys:
            k[int(table[b, j // 64]), :, j % 64, 3] = -math.inf
    want, spread = pu.attention(q, k, v, table, pos)
    assert np.isnan(want[2, 0]).all() and np.isfinite(want[:2]).all() and np.isfinite(want[2, 1:]).all()
    check(attend(q, k, v, table, pos), want, spread, [T] * B)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,n", [(1, 900), (130, 900)])
def test_scores_of_any_finite_size(d, T, n):
    """Products of 1e3 to 1e37 of both signs, exact in fp32: one key leads or two tie, and the next is
    a thirtieth of a score behind: it weighs something at 1e3 alone."""
    g = gen(d)
    sizes = [1e3, 1e5, 1e8, 1e12, 1e20, 1e37]
    B, G = len(sizes), 2
    q, k, v, table, pos = problem(g, B, T, 1, G, d, 32, [n] * B, [T] * B)
    q.zero_()
    k[torch.isfinite(k)] = 0.0
    for b, s in enumerate(sizes):
        q[b, ..., 5] = s / 30 * (1 + torch.rand(T, G, generator=g)).to(bf16)
        q[b, :, 1, 5] *= -1
        for j in range(n):
            k[int(table[b, j // 32]), :, j % 32, 5] = float(torch.randint(-29, 30, (1,), generator=g))
        for j, x in ((int(torch.randint(0, n - T, (1,), generator=g)), 30.0), (int(torch.randint(0, n - T, (1,), generator=g)), -30.0)):
            k[int(table[b, j // 32]), :, j % 32, 5] = x
        if b % 2:
            k[int(table[b, 700 // 32]), :, 700 % 32, 5] = 30.0
    want, spread = pu.attention(q, k, v, table, pos)
    check(attend(q, k, v, table, pos), want, spread, [T] * B)


@pytest.mark.parametrize("scale", [1e-30, 0.01, 1.0, 7.5])
def test_scale(scale):
    g = gen(2)
    p = problem(g, 2, 20, 2, 4, 64, 16, [150, 20], [20, 20], std=0.4)
    want, spread = pu.attention(*p, None, 0, 0, scale)
    check(attend(*p, None, 0, 0, scale), want, spread, [20, 20])


def test_attend_strides_of_q():
    """q as a slice of a projection, heads outermost, one for the whole batch, one for all heads, and
    strides of dimensions of size 1 that are any numbers."""
    g = gen(8)
    B, T, H_kv, G, d = 3, 30, 2, 4, 128
    q, k, v, table, pos = problem(g, B, T, H_kv, G, d, 64, [200, 30, 129], [T] * 3)
    fused = torch.cat((rand(g, B, T, 3, d), q, rand(g, B, T, 2, d)), 2).to(DEV)
    for x in (fused[:, :, 3:11], q.transpose(1, 2).contiguous().transpose(1, 2).to(DEV), q[:1].to(DEV).expand(B, T, 8, d),
              q[:, :, :1].to(DEV).expand(B, T, 8, d), q[:, :1].to(DEV).expand(B, T, 8, d)):
        want, spread = pu.attention(x.cpu(), k, v, table, pos)
        check(attend(x, k, v, table, pos), want, spread, [T] * 3)
    one = torch.as_strided(q.to(DEV).contiguous(), (1, 1, 8, 128), (7, 3, 128, 1))
    want, spread = pu.attention(q[:1, :1], k, v, table[:1], [150])
    check(attend(one, k, v, table[:1], [150]), want, spread, [1])


def test_a_page_outside_the_pool_counts_as_zeros():
    g = gen(4)
    q, k, v, table, pos = problem(g, 3, 6, 2, 4, 64, 16, [100, 300, 40], [6] * 3)
    table[0, 2], table[1, 0], table[1, 17] = k.shape[0], -5, 1 << 30
    ws = santa.new_workspace(64 << 20, DEV)
    want, spread = pu.attention(q, k, v, table, pos)
    got = attend(q, k, v, table, pos, workspace=ws)
    assert santa.device_status(ws) == santa.DEV_BAD_PAGE
    check(got, want, spread, [6] * 3)
    # an entry that no visible key needs is not looked at
    got = attend(q[2:], k, v, torch.cat((table[2:], table[:1]), 1)[:, :19], pos[2:], workspace=ws)
    assert santa.device_status(ws) == 0
    check(got, want[2:], spread[2:], [6])


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("T", [1, 70])
def test_pages_before_the_window_may_be_gone(page, T):
    """A cache that gives back the pages behind the window: their entries name no page, and no error is
    reported; one page fewer, and it is."""
    g = gen(page + T)
    n, window, sinks = 1300, 200, 5
    q, k, v, table, pos = problem(g, 2, T, 2, 4, 64, page, [n, n - 100], [T, T])
    want, spread = pu.attention(q, k, v, table, pos, None, window, sinks)
    ws = santa.new_workspace(64 << 20, DEV)
    lowest = [pos[b] - window + 1 for b in range(2)]
    for b in range(2):
        table[b, -(-sinks // page):lowest[b] // page] = -1
    check(attend(q, k, v, table, pos, None, window, sinks, workspace=ws), want, spread, [T, T])
    assert santa.device_status(ws) == 0
    table[1, lowest[1] // page] = k.shape[0]
    attend(q, k, v, table, pos, None, window, sinks, workspace=ws)
    assert santa.device_status(ws) == santa.DEV_BAD_PAGE


@pytest.mark.parametrize("B,T,H_kv,G,d,page,lengths,window", [
    (1, 1, 8, 4, 128, 64, [100003], 0), (3, 1, 8, 4, 128, 128, [30011, 1, 9000], 0), (1, 7, 4, 8, 64, 16, [50001], 0),
    (1, 33, 2, 4, 128, 32, [20000], 0), (2, 300, 4, 4, 128, 64, [5000, 300], 0), (4, 100, 2, 8, 64, 16, [3000, 100, 101, 1777], 333),
    (1, 600, 1, 2, 128, 256, [4096], 0), (7, 65, 2, 4, 128, 16, [65, 70, 1000, 129, 128, 257, 4000], 0),
])
def test_the_same_bits_every_time(B, T, H_kv, G, d, page, lengths, window):
    """Forty calls each, cold and warm caches in turn, on one workspace: no wait runs out, no piece is
    missed, no bit differs."""
    g = gen(B + T)
    q, k, v, table = big(g, B, T, H_kv, G, d, page, lengths, T + d)
    pos = ints([n - min(T, n) for n in lengths])
    counts = ints([min(T, n) for n in lengths])
    cache = santa.PagedCache(k, v, table.to(DEV))
    ws = santa.new_workspace(64 << 20, DEV)
    flush = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)
    first = None
    for i in range(40):
        if i % 2:
            flush.fill_(i)
        out = torch.full_like(q, 3.0)
        santa.attend_paged(q, cache, pos, counts, window, 4, out=out, workspace=ws)
        if first is None:
            first = out
            assert torch.isfinite(out).all()
        assert torch.equal(out, first)
    assert santa.device_status(ws) == 0


def test_calls_on_two_streams_at_once():
    """Calls without a workspace of their own, on two streams, each many times over."""
    g = gen(20)
    q, k, v, table = big(g, 2, 40, 2, 4, 128, 64, [3000, 2000], 5)
    cache, pos = santa.PagedCache(k, v, table.to(DEV)), ints([2960, 1960])
    want = santa.attend_paged(q, cache, pos)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            outs[i].append(santa.attend_paged(q, cache, pos, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for row in outs for o in row)


def test_positions_out_of_range_skip_the_row():
    g = gen(6)
    q, k, v, table, pos = problem(g, 6, 4, 1, 4, 64, 16, [50] * 6, [4] * 6)
    want, spread = pu.attention(q, k, v, table, pos)
    n_max = table.shape[1] * 16
    ws = santa.new_workspace(64 << 20, DEV)
    out = torch.full((6, 4, 4, 64), 7.0, dtype=bf16, device=DEV)
    pos[1], pos[2], pos[3], pos[5] = -1, n_max - 3, (1 << 31) - 1, 46
    counts = [4, 4, 4, 2, 5, 4]
    attend(q, k, v, table, pos, counts, out=out, workspace=ws)
    assert santa.device_status(ws) == santa.DEV_BAD_POSITION
    assert (out[1:5] == 7).all()
    check(out[[0, 5]], want[[0, 5]], spread[[0, 5]], [4, 4])
    assert santa.device_status(ws) == 0


def reference_on_gpu(q, k, v, table, pos, window, sinks, b, rows):
    """float64 result and spread of tokens `rows` of sequence b, on the GPU."""
    d, H_kv = q.shape[3], k.shape[1]
    n = pos[b] + max(rows) + 1
    pages = table[b, :-(-n // k.shape[2])].long().to(DEV)
    kb, vb = (x[pages].transpose(1, 2).flatten(0, 1)[:n].double() for x in (k, v))     # [n, H_kv, d]
    outs, spreads = [], []
    for t in rows:
        j = torch.arange(n, device=DEV)
        seen = j <= pos[b] + t
        if window:
            seen &= (j > pos[b] + t - window) | (j < sinks)
        s = torch.einsum("hgd,nhd->hgn", q[b, t].double().view(H_kv, -1, d), kb) / math.sqrt(d)
        w = torch.softmax(s.masked_fill(~seen, -math.inf), -1)
        o = torch.einsum("hgn,nhd->hgd", w, vb)
        sp = torch.stack([torch.einsum("gn,ngd->gd", w[h], (vb[:, h, None] - o[h]).abs()) for h in range(H_kv)])
        outs.append(o.flatten(0, 1))
        spreads.append(sp.flatten(0, 1))
    return f64(torch.stack(outs)), f64(torch.stack(spreads))


def big(g, B, T, H_kv, G, d, page, lengths, seed):
    cols = -(-max(lengths) // page)
    table, n_pages = pu.pages(g, lengths, page, cols)
    dg = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(B, T, H_kv * G, d, generator=dg, device=DEV)
    q = (3 * math.sqrt(d) * x / x.norm(dim=-1, keepdim=True)).to(bf16)
    k, v = (torch.randn(n_pages, H_kv, page, d, generator=dg, device=DEV, dtype=torch.float32).to(bf16) for _ in range(2))
    return q, k, v, table


@pytest.mark.parametrize("B,T,H_kv,G,d,page,lengths,window,sinks", [
    (1, 1, 8, 4, 128, 64, [100003], 0, 0),
    (1, 3, 2, 8, 64, 16, [131071], 0, 0),
    (5, 1, 8, 4, 128, 128, [40000, 1, 129, 33333, 20000], 0, 0),
    (4, 2, 4, 2, 64, 256, [30000, 2, 50001, 777], 4097, 5),
    (1, 2048, 2, 4, 128, 64, [9000], 0, 0),
    (2, 1500, 2, 8, 128, 16, [1500, 6001], 1000, 100),
    (1, 4099, 1, 1, 64, 32, [20000], 0, 0),
    (64, 9, 2, 4, 64, 64, [100 + 97 * i for i in range(64)], 0, 0),
    (1, 1, 1, 8, 64, 256, [524288], 0, 0),                                    # the longest cache
    (1024, 1, 1, 4, 64, 16, [1 + (i * 7) % 53 for i in range(1024)], 0, 0),   # the most rows
    (1000, 40, 1, 4, 64, 16, [(i * 7) % 41 for i in range(1000)], 0, 0),      # padded, rows of no length among them
    (2, 4096, 1, 4, 64, 64, [5, 4100], 0, 0),                                 # padded: few tokens of a long chunk
])
def test_attend_at_length(B, T, H_kv, G, d, page, lengths, window, sinks):
    """Work that spans many CTAs: tokens of every sequence against 64 bits on the GPU; the same call
    twice gives the same bits."""
    g = gen(T + d)
    q, k, v, table = big(g, B, T, H_kv, G, d, page, lengths, T)
    pos = [n - min(T, n) for n in lengths]
    counts = [min(T, n) for n in lengths]
    cache = santa.PagedCache(k, v, table.to(DEV))
    ws = santa.new_workspace(64 << 20, DEV)
    out = santa.attend_paged(q, cache, ints(pos), ints(counts), window, sinks, workspace=ws)
    assert santa.device_status(ws) == 0
    assert torch.equal(out, santa.attend_paged(q, cache, ints(pos), ints(counts), window, sinks, workspace=ws))
    for b in list(range(B))[:: max(1, B // 8)]:
        c = counts[b]
        if c == 0:
            continue
        rows = sorted({0, c - 1, c // 2, c // 3, min(c - 1, 63), min(c - 1, 64), min(c - 1, 257)})
        want, spread = reference_on_gpu(q, k, v, table, pos, window, sinks, b, rows)
        check(out[b, rows][None], want[None], spread[None], [len(rows)])


def test_the_result_may_go_over_the_queries():
    """out = q: every row of a tile is read before the tile's results are written."""
    g = gen(21)
    q, k, v, table = big(g, 2, 300, 2, 4, 128, 64, [5000, 300], 9)
    cache, pos = santa.PagedCache(k, v, table.to(DEV)), ints([4700, 0])
    want = santa.attend_paged(q, cache, pos)
    for _ in range(5):
        x = q.clone()
        assert santa.attend_paged(x, cache, pos, out=x) is x
        assert torch.equal(x, want)


def test_pool_rows_beyond_32_bits():
    """Pages whose elements lie beyond 2^31: written, read and attended to."""
    H_kv, page, d, T = 4, 64, 128, 70
    n_pages = (1 << 31) // (H_kv * page * d) + 40
    k, v = (torch.empty(n_pages, H_kv, page, d, dtype=bf16, device=DEV) for _ in range(2))
    table = ints([[n_pages - 1, n_pages - 3, 0, n_pages - 39]])
    g = gen(7)
    new_k, new_v, q = rand(g, 1, 230, H_kv, d), rand(g, 1, 230, H_kv, d), rand(g, 1, T, 8, d)
    cache = santa.PagedCache(k, v, table)
    santa.paged_append(cache, new_k.to(DEV), new_v.to(DEV), ints([0]))
    assert torch.equal(k[n_pages - 3, :, 5].cpu(), new_k[0, 69]) and torch.equal(v[n_pages - 39, :, 37].cpu(), new_v[0, 229])
    got = santa.attend_paged(q.to(DEV), cache, ints([160]))
    some = torch.tensor([n_pages - 1, n_pages - 3, 0, n_pages - 39])
    want, spread = pu.attention(q, k[some].cpu(), v[some].cpu(), torch.arange(4)[None], [160])
    check(got, want, spread, [T])


# ------------------------------------------------------------------ together

def contiguous(cache, n_max):
    """The bf16 cache [B, H_kv, n_max, d] of the decode calls."""
    return [x[cache.table.long().clamp(min=0)].transpose(2, 3).flatten(1, 2).transpose(1, 2)[:, :, :n_max].contiguous()
            for x in (cache.k, cache.v)]


@pytest.mark.parametrize("d,G,page,layout", [(128, 4, 64, "halves"), (64, 2, 16, "pairs")])
def test_prompts_in_chunks_then_decode_steps(d, G, page, layout):
    """Ragged prompts in chunks of 48, then single tokens: every result as from one pass over the
    rotated whole, and the last steps as decode() and decode_window() have them over a contiguous copy."""
    g = gen(d)
    B, H_kv, total, chunk = 3, 2, 170, 48
    H_q = H_kv * G
    lens = [170, 101, 49]
    qkv = rand(g, B, total, H_q + 2 * H_kv, d)
    t = santa.rope_table(d, 500000.0, layout, "bands", 8.0, original=64)
    f, _ = pu.frequencies(d, 500000.0, "bands", 8.0, original=64)
    cols = -(-(total + 8) // page)
    table, n_pages = pu.pages(g, [n + 8 for n in lens], page, cols)
    cache = santa.new_paged_cache(n_pages, H_kv, page, d, B, cols)
    cache.table.copy_(table)
    pos = ints([0] * B)
    rot_q, rot_k = (torch.from_numpy(pu.rotate(x, f, 1.0, layout, [0] * B)).to(bf16) for x in qkv.split((H_q, 2 * H_kv), 2))
    v = qkv[:, :, H_q + H_kv:]
    # the reference over the whole, one page a sequence
    pool_k, pool_v = rot_k[:, :, :H_kv].transpose(1, 2), v.transpose(1, 2)
    want, spread = pu.attention(rot_q, pool_k.contiguous(), pool_v.contiguous(), torch.arange(B)[:, None], [0] * B, lens)
    at = 0
    while at < total:
        counts = ints([max(0, min(chunk, n - at)) for n in lens])
        q, k_new, v_new = qkv[:, at:at + chunk].to(DEV).split((H_q, H_kv, H_kv), 2)
        q = santa.paged_append(cache, k_new, v_new, pos, counts, rope=t, q=q)
        out = santa.attend_paged(q, cache, pos, counts)
        for b in range(B):
            c = int(counts[b])
            # q and K may differ from the reference's by a rounding where theirs is near a border
            assert np.abs(f64(out)[b, :c] - want[b, at:at + c]).max(initial=0) <= \
                (2 * pu.tolerance(want[b, at:at + c], spread[b, at:at + c])).max(initial=0) + 2.0 ** -6
        pos += counts
        at += chunk
    assert pos.tolist() == lens
    for _ in range(4):
        q, k_new, v_new = rand(g, B, 1, H_q + 2 * H_kv, d).to(DEV).split((H_q, H_kv, H_kv), 2)
        q = santa.paged_append(cache, k_new, v_new, pos, rope=t, q=q)
        out = santa.attend_paged(q, cache, pos)
        near = santa.attend_paged(q, cache, pos, window=40, sinks=3)
        pos += 1
        k_all, v_all = contiguous(cache, total + 8)
        dense, _ = santa.decode(q[:, 0].contiguous(), k_all, v_all, pos, 1, "dense")
        windowed = santa.decode_window(q[:, 0].contiguous(), k_all, v_all, pos, 40, 3)
        for got, ref in ((out, dense), (near, windowed)):
            # roundings of the weights and of the result against none
            assert (got[:, 0].float() - ref).abs().max() <= 2.0 ** -7 * v_all.abs().max()


def test_rope_feeds_the_other_caches():
    """santa.rope before kv4_append and decode_kv4: the 4-bit cache holds the rotated keys."""
    g = gen(12)
    B, T, H_kv, d = 2, 50, 2, 64
    k, v = rand(g, B, T, H_kv, d).to(DEV), rand(g, B, T, H_kv, d).to(DEV)
    t = santa.rope_table(d)
    rotated = santa.rope(k, t, ints([0, 0]))
    a, b = santa.new_kv4_cache(B, H_kv, 64, d), santa.new_kv4_cache(B, H_kv, 64, d)
    santa.kv4_append(a, rotated, v, ints([0, 0]))
    room = torch.empty_like(k)
    santa.rope(k, t, ints([0, 0]), out=room)
    santa.kv4_append(b, room, v, ints([0, 0]))
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    q = santa.rope(rand(g, B, 1, 8, d).to(DEV), t, ints([T - 1, T - 1]))
    assert torch.isfinite(santa.decode_kv4(q[:, 0].contiguous(), a, ints([T, T]))).all()


def test_captured_steps_and_two_graphs_at_once():
    """A captured decode step (append, attend, advance) replayed as a loop, against the same steps
    made eagerly; two graphs of different shapes replayed on two streams at once."""
    g = gen(13)
    B, H_kv, G, d, page, cols = 2, 2, 4, 128, 16, 30
    H_q = H_kv * G
    t = santa.rope_table(d)
    steps = rand(g, 20, B, 1, H_q + 2 * H_kv, d).to(DEV)
    table = torch.randperm(B * cols, generator=g).view(B, cols).to(torch.int32).to(DEV)
    base_k, base_v = rand(g, B * cols, H_kv, page, d).to(DEV), rand(g, B * cols, H_kv, page, d).to(DEV)

    def step(cache, qkv, pos):
        q, k, v = qkv.split((H_q, H_kv, H_kv), 2)
        out = santa.attend_paged(santa.paged_append(cache, k, v, pos, rope=t, q=q), cache, pos)
        pos += 1
        return out

    eager = santa.PagedCache(base_k.clone(), base_v.clone(), table)
    pos = ints([440, 100])
    want = [step(eager, x, pos).clone() for x in steps]

    caches = [santa.PagedCache(base_k.clone(), base_v.clone(), table) for _ in range(2)]
    graphs, ins, outs, poss = [], [], [], []
    for c in caches:
        x, p = steps[0].clone(), ints([440, 100])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o = step(c, x, p)
        graphs.append(graph), ins.append(x), outs.append(o), poss.append(p)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for x in steps:
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                ins[i].copy_(x)
                graphs[i].replay()
                got[i].append(outs[i].clone())
    torch.cuda.synchronize()
    for i in range(2):
        assert poss[i].tolist() == [460, 120]
        assert all(torch.equal(a, b) for a, b in zip(got[i], want))
        assert torch.equal(caches[i].k, eager.k) and torch.equal(caches[i].v, eager.v)


def test_explicit_streams():
    """Each call on a stream of its own, without one of the caller's being current."""
    g = gen(14)
    q, k, v, table, pos = problem(g, 2, 40, 2, 4, 64, 32, [300, 40], [40, 40])
    want, spread = pu.attention(q, k, v, table, pos)
    cache = santa.PagedCache(k.to(DEV), v.to(DEV), table.to(DEV))
    qd, pd = q.to(DEV), ints(pos)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = santa.attend_paged(qd, cache, pd, stream=s)
    t = santa.rope_table(64)
    torch.cuda.synchronize()
    r = santa.rope(qd, t, pd, stream=s)
    new = rand(g, 2, 1, 2, 64).to(DEV)
    torch.cuda.synchronize()
    santa.paged_append(cache, new, new, pd, stream=s)
    s.synchronize()
    check(out, want, spread, [40, 40])
    f, _ = pu.frequencies(64)
    check_rope(r, q, f, 1.0, "halves", pos, [40, 40], r)
    for b in range(2):
        assert torch.equal(cache.v[int(table[b, pos[b] // 32]), :, pos[b] % 32], new[b, 0])


def test_refusals_of_the_binding():
    g = gen(1)
    q, k, v, table, pos = problem(g, 2, 3, 2, 4, 64, 16, [30, 30], [3, 3])
    cache = santa.PagedCache(k.to(DEV), v.to(DEV), table.to(DEV))
    qd, pd, t = q.to(DEV), ints(pos), santa.rope_table(64)
    new = rand(g, 2, 3, 2, 64).to(DEV)
    for call in (lambda: santa.attend_paged(qd.float(), cache, pd), lambda: santa.attend_paged(qd[:1], cache, pd),
                 lambda: santa.attend_paged(qd[..., ::2], cache, pd), lambda: santa.attend_paged(qd, cache, pd.long()),
                 lambda: santa.attend_paged(qd, cache, pd[:1]), lambda: santa.attend_paged(qd, cache, pd, pd[:1]),
                 lambda: santa.attend_paged(qd, cache._replace(table=cache.table.long()), pd),
                 lambda: santa.attend_paged(qd, cache._replace(k=cache.k.float()), pd),
                 lambda: santa.attend_paged(qd, cache._replace(v=cache.v[:-1]), pd),
                 lambda: santa.attend_paged(qd, cache, pd, out=torch.empty_like(qd, dtype=torch.float32)),
                 lambda: santa.attend_paged(qd, cache, pd, out=torch.empty(2, 8, 3, 64, dtype=bf16, device=DEV).transpose(1, 2)),
                 lambda: santa.attend_paged(qd, cache, pd, window=1 << 31),
                 lambda: santa.paged_append(cache, new[:, :2], new, pd), lambda: santa.paged_append(cache, new, new[:, :, :1], pd),
                 lambda: santa.paged_append(cache, new, new, pd, q=qd), lambda: santa.paged_append(cache, new, new, pd, q_out=qd),
                 lambda: santa.paged_append(cache, new, new, pd, rope=t, q=qd, q_out=qd[:, :2]),
                 lambda: santa.rope(qd, t._replace(turns=t.turns[:-1]), pd), lambda: santa.rope(qd, t._replace(layout="x"), pd),
                 lambda: santa.rope(qd, t, pd.float()), lambda: santa.rope(qd, t, pd, out=qd[:, :2])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: santa.attend_paged(qd, cache, pd, window=-1), lambda: santa.attend_paged(qd, cache, pd, scale=-1.0),
                 lambda: santa.attend_paged(qd, cache, pd, workspace=torch.zeros(256, dtype=torch.uint8, device=DEV)),
                 lambda: santa.rope(qd, santa.rope_table(128), pd), lambda: santa.rope(qd, santa.rope_table(8), pd),
                 lambda: santa.rope(qd[:, :, :1].expand(2, 3, 8, 64), t, pd, out=qd[:, :, :1].expand(2, 3, 8, 64)),
                 lambda: santa.attend_paged(qd[:, :, :3], cache, pd)):
        with pytest.raises(santa.SantaError):
            call()
    assert santa.rope(qd[:, :0], t, pd).shape == (2, 0, 8, 64)
    assert santa.attend_paged(qd[:, :0], cache, pd).shape == (2, 0, 8, 64)
    assert santa.paged_append(cache, new[:, :0], new[:, :0], pd) is None
