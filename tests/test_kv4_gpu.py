"""The 4-bit KV cache and windowed exact attention on the GPU, against tests/kv4_util.py (the
definitions in 64 bits).  Codes, scales and rows read back are compared bit for bit.

Tolerance of attention outputs (fp32, before any rounding to bf16): a relative error e in
each weight moves sum p v by at most 2 e max|v|.  A score is a sum of d exact products added
in steps of 16 in fp32: at most (d/16 + 2) roundings of 2^-23 (the tensor cores truncate)
of sum |q_i k_i| sigma, which the inputs here keep below 40 on average, so e <= 10 * 2^-23 * 40
= 5e-5; exponential, weights and sums add a few 2^-21.  2 e max|v| is 1e-4 max|v|.
"""
import numpy as np
import pytest
import torch

from stochastic_sparse_kv_gb300 import santa, workloads
from tests import kv4_util

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = 1e-4
NAN = float("nan")
# what a group of ones holds: its scale is the 4-bit number nearest 1/6 = 0.16667 between
# 10/64 (off by 0.01042) and 11/64 (off by 0.00521), and 64/11 = 5.8 is nearest 6
ONE = 6 * 11 / 64


@pytest.fixture(scope="module", autouse=True)
def _lib():
    santa.load()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rand(g, *shape):
    return torch.randn(*shape, generator=g).to(torch.bfloat16)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def filled_cache(k, v):
    """A cache that holds the quantised k, v [B, H_kv, n, d] (CPU bf16), by the reference."""
    parts = [torch.from_numpy(x).to(DEV) for t in (k, v) for x in kv4_util.quantise(t)]
    return santa.KV4Cache(*parts)


def held(cache):
    k, ks, v, vs = (x.cpu().numpy() for x in cache)
    return kv4_util.values(k, ks), kv4_util.values(v, vs)


# ------------------------------------------------------------------ writing and reading

@pytest.mark.parametrize("d,H_kv,T,n_max", [(128, 8, 1, 32), (64, 1, 1, 16), (128, 1, 17, 48), (64, 5, 33, 64),
                                            (128, 3, 333, 512), (64, 2, 1000, 1008)])
def test_append_and_read_bit_exact(d, H_kv, T, n_max):
    g = gen(d + T)
    B = 3
    k, v = rand(g, B, T, H_kv, d) * 3, rand(g, B, T, H_kv, d) * 0.01
    pos = [0, n_max - T, (n_max - T) // 2]
    cache = santa.new_kv4_cache(B, H_kv, n_max, d)
    for t in cache:
        t.fill_(0xA5)
    want = [x.cpu().numpy().copy() for x in cache]
    for i, src in ((0, k), (2, v)):
        c, s = kv4_util.quantise(src.transpose(1, 2).contiguous())
        for b in range(B):
            want[i][b, :, pos[b]:pos[b] + T] = c[b]
            want[i + 1][b, :, pos[b]:pos[b] + T] = s[b]
    santa.kv4_append(cache, k.to(DEV), v.to(DEV), ints(pos))
    for got, w in zip(cache, want):
        assert np.array_equal(got.cpu().numpy(), w)      # the new rows, and every other byte as it was
    ko, vo = (torch.full((B, T, H_kv, d), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    santa.kv4_read(cache, ints(pos), ko, vo)
    for got, i in ((ko, 0), (vo, 2)):
        for b in range(B):
            ref = kv4_util.values(want[i][b, :, pos[b]:pos[b] + T], want[i + 1][b, :, pos[b]:pos[b] + T])
            assert np.array_equal(got[b].transpose(0, 1).cpu().double().numpy(), ref)


@pytest.mark.parametrize("d", [64, 128])
def test_ragged_counts_and_strides(d):
    """K and V as head slices of one projection, source heads outermost, and one prompt
    broadcast to every batch row; counts 0, 1, T and between; rows past a count stay."""
    g = gen(d)
    B, T, H_kv, n_max = 4, 21, 4, 64
    pos, counts = [5, 0, 43, 10], [21, 0, 20, 1]
    qkv = rand(g, B, T, 6 * H_kv, d).to(DEV)
    headmajor = rand(g, B, H_kv, T, d).to(DEV).transpose(1, 2)
    one = rand(g, 1, T, H_kv, d).to(DEV).expand(B, T, H_kv, d)
    for k, v in ((qkv[:, :, 4 * H_kv:5 * H_kv], qkv[:, :, 5 * H_kv:]), (headmajor, one)):
        cache = santa.new_kv4_cache(B, H_kv, n_max, d)
        for t in cache:
            t.fill_(0x11)
        want = [x.cpu().numpy().copy() for x in cache]
        for i, src in ((0, k), (2, v)):
            c, s = kv4_util.quantise(src.cpu().transpose(1, 2).contiguous())
            for b in range(B):
                want[i][b, :, pos[b]:pos[b] + counts[b]] = c[b, :, :counts[b]]
                want[i + 1][b, :, pos[b]:pos[b] + counts[b]] = s[b, :, :counts[b]]
        santa.kv4_append(cache, k, v, ints(pos), ints(counts))
        for got, w in zip(cache, want):
            assert np.array_equal(got.cpu().numpy(), w)
        # read into a bf16 cache of another capacity (head-major) and into token-major rows
        kc = torch.full((B, H_kv, n_max + 3, d), 9.0, dtype=torch.bfloat16, device=DEV)
        vo = torch.full((B, T, H_kv, d), 9.0, dtype=torch.bfloat16, device=DEV)
        santa.kv4_read(cache, ints(pos), kc.transpose(1, 2)[:, :T], vo, ints(counts))
        kv_, vv = held(cache)
        for b in range(B):
            c, p = counts[b], pos[b]
            assert np.array_equal(kc[b, :, :c].cpu().double().numpy(), kv_[b, :, p:p + c])
            assert torch.all(kc[b, :, c:] == 9)
            assert np.array_equal(vo[b, :c].transpose(0, 1).cpu().double().numpy(), vv[b, :, p:p + c])
            assert torch.all(vo[b, c:] == 9)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shift,pad", [(8, 0), (0, 8), (8, 8), (16, 16), (24, 0)])
def test_rows_aligned_to_16_bytes_only(d, shift, pad):
    """K and V at 16-byte offsets of their own, head strides that are odd multiples of 8."""
    g = gen(shift + pad)
    B, T, H_kv, n_max = 2, 19, 3, 32
    room = rand(g, B, T, H_kv, d + pad).to(DEV).reshape(-1)

    def rows_at(offset):
        buf = torch.full((offset + room.numel() + 32,), 3.0, dtype=torch.bfloat16, device=DEV)
        buf[offset:offset + room.numel()] = room
        return torch.as_strided(buf, (B, T, H_kv, d), (T * H_kv * (d + pad), H_kv * (d + pad), d + pad, 1), offset), buf

    (k, _), (v, _) = rows_at(shift), rows_at(0)
    cache = santa.new_kv4_cache(B, H_kv, n_max, d)
    santa.kv4_append(cache, k, v, ints([3, 13]))
    c, s = kv4_util.quantise(k.cpu().transpose(1, 2).contiguous())
    for b, p in ((0, 3), (1, 13)):
        for got in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
            assert np.array_equal(got[0][b, :, p:p + T].cpu().numpy(), c[b])
            assert np.array_equal(got[1][b, :, p:p + T].cpu().numpy(), s[b])
    (ko, kbuf), (vo, vbuf) = rows_at(shift), rows_at(0)
    before = kbuf.clone()
    santa.kv4_read(cache, ints([3, 13]), ko, vo)
    ref = kv4_util.values(c, s)
    assert np.array_equal(ko.cpu().transpose(1, 2).double().numpy(), ref)
    assert np.array_equal(vo.cpu().transpose(1, 2).double().numpy(), ref)
    ko.copy_(k)
    assert torch.equal(kbuf, before)          # nothing beside the rows was written


@pytest.mark.parametrize("d", [64, 128])
def test_as_many_tokens_as_there_may_be(d):
    """2^31 - 1 groups, or the most below: one prompt of which few tokens are live, its token stride 0."""
    T = ((1 << 31) - 1) // (d // 16)
    row = rand(gen(d), 1, 1, 1, d).to(DEV)
    cache = santa.new_kv4_cache(1, 1, 16, d)
    santa.kv4_append(cache, row.expand(1, T, 1, d), row.expand(1, T, 1, d), ints([6]), ints([3]))
    c, s = kv4_util.quantise(row.cpu())
    for codes, scales in (cache[:2], cache[2:]):
        live = np.zeros(16, dtype=bool)
        live[6:9] = True
        assert np.array_equal(codes[0, 0, 6:9].cpu().numpy(), np.repeat(c.reshape(1, -1), 3, 0))
        assert np.array_equal(scales[0, 0, 6:9].cpu().numpy(), np.repeat(s.reshape(1, -1), 3, 0))
        assert not codes[0, 0, ~live].any() and not scales[0, 0, ~live].any()


def test_strides_of_single_dimensions_are_not_read():
    """One row of one head, its batch, token and head strides any numbers."""
    g = gen(3)
    room = rand(g, 2, 128).to(DEV)
    k, v = (torch.as_strided(room, (1, 1, 1, 128), st, 128 * i) for i, st in enumerate([(0, 0, 0, 1), (7, 3, 1, 1)]))
    cache = santa.new_kv4_cache(1, 1, 16, 128)
    santa.kv4_append(cache, k, v, ints([5]))
    out = torch.zeros(3, 128, dtype=torch.bfloat16, device=DEV)
    ko, vo = (torch.as_strided(out, (1, 1, 1, 128), st, 128 * i) for i, st in enumerate([(1, 5, 0, 1), (0, 0, 0, 1)]))
    santa.kv4_read(cache, ints([5]), ko, vo)
    ref = kv4_util.values(*kv4_util.quantise(room.cpu()))
    assert np.array_equal(out[:2].cpu().double().numpy(), ref) and torch.all(out[2] == 0)


def test_every_largest_magnitude_and_every_quotient():
    """Every finite bf16 as a group's largest magnitude (all scales, ties and the ends of the
    range), beside values of all smaller sizes; and every bf16 mantissa against every scale
    mantissa near all seven borders of the grid."""
    top = torch.arange(0x7F80, dtype=torch.int16).view(torch.bfloat16)      # 0 .. largest finite
    g = gen(0)
    x = torch.zeros(len(top), 16, dtype=torch.bfloat16)
    frac = (torch.rand(len(top), 15, generator=g) * 2 - 1)
    x[:, 0] = top
    x[:, 1:] = (top.float().unsqueeze(1) * frac).to(torch.bfloat16)
    m = torch.arange(128, 256).float()                                      # 8-bit mantissas
    near = torch.cat([(m * 2.0 ** e).to(torch.bfloat16) for e in range(-10, -4)])
    groups = []
    for a in range(8, 16):                                                  # the scale's mantissa
        y = near[near <= a * 6 / 8]
        y = torch.cat([y, torch.zeros(-len(y) % 15)]).view(-1, 15)
        groups.append(torch.cat([torch.full((len(y), 1), a * 6 / 8), y], 1))
    x = torch.cat([x, torch.cat(groups).to(torch.bfloat16)])
    x = torch.cat([x, torch.zeros(-len(x) % 8, 16, dtype=torch.bfloat16)]).view(1, -1, 1, 128)
    T = x.shape[1]
    cache = santa.new_kv4_cache(1, 1, T, 128)
    santa.kv4_append(cache, x.to(DEV), -x.to(DEV), ints([0]))
    for got, src in (((cache.k, cache.k_scale), x), ((cache.v, cache.v_scale), -x)):
        c, s = kv4_util.quantise(src.transpose(1, 2).contiguous())
        assert np.array_equal(got[1][:, :, :T].cpu().numpy(), s)
        assert np.array_equal(got[0][:, :, :T].cpu().numpy(), c)


def test_groups_with_nan_or_infinity_read_back_as_nan():
    x = torch.ones(1, 2, 1, 64, dtype=torch.bfloat16)
    x[0, 0, 0, 3], x[0, 0, 0, 40], x[0, 1, 0, 63] = NAN, float("-inf"), float("inf")
    cache = santa.new_kv4_cache(1, 1, 16, 64)
    santa.kv4_append(cache, x.to(DEV), x.to(DEV), ints([2]))
    k, v = (torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    santa.kv4_read(cache, ints([2]), k, v)
    bad = torch.zeros(1, 2, 1, 64, dtype=torch.bool)
    bad[0, 0, 0, :16] = bad[0, 0, 0, 32:48] = bad[0, 1, 0, 48:] = True
    for t in (k, v):
        assert torch.equal(torch.isnan(t.cpu()), bad) and torch.all(t.cpu()[~bad] == ONE)


def test_reading_every_code_and_scale():
    codes = torch.arange(16, dtype=torch.uint8)
    row = (codes[0::2] | (codes[1::2] << 4)).repeat(8)                       # 8 groups of all 16 codes
    cache = santa.new_kv4_cache(1, 1, 32, 128)
    cache.k.copy_(row.to(DEV).expand(1, 1, 32, 64))
    cache.k_scale.copy_(torch.arange(256, dtype=torch.uint8).view(1, 1, 32, 8).to(DEV))
    k, v = (torch.zeros(1, 32, 1, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    santa.kv4_read(cache, ints([0]), k, v)
    ref = kv4_util.values(cache.k.cpu().numpy(), cache.k_scale.cpu().numpy())[0, 0]
    got = k[0, :, 0].cpu().double().numpy()
    # scales above 10240 are never written: 6 of them may exceed fp16, and they need not be exact
    assert np.array_equal(got[:28], ref[:28])
    assert np.array_equal(got[28].reshape(8, 16)[:3], ref[28].reshape(8, 16)[:3])
    assert np.isnan(got[31].reshape(8, 16)[7]).all()


def test_rows_outside_the_cache_are_skipped_and_reported():
    B, T, n_max = 5, 4, 16
    pos, counts = [13, -1, 0, 12, 2], [4, 1, 5, 4, -2]     # only row 3 is inside
    x = torch.ones(B, T, 1, 64, dtype=torch.bfloat16, device=DEV)
    ws = santa.new_workspace(65536, DEV)
    cache = santa.new_kv4_cache(B, 1, n_max, 64)
    santa.kv4_append(cache, x, x, ints(pos), ints(counts), workspace=ws)
    assert santa.device_status(ws) == santa.DEV_BAD_POSITION and santa.device_status(ws) == 0
    live = (cache.k_scale.sum((1, 3)) != 0).cpu()
    want = torch.zeros(B, n_max, dtype=torch.bool)
    want[3, 12:] = True
    assert torch.equal(live, want)
    y = torch.full_like(x, 5.0)
    santa.kv4_read(cache, ints(pos), y, y.clone(), ints(counts), workspace=ws)
    assert santa.device_status(ws) == santa.DEV_BAD_POSITION
    assert torch.all(y[[0, 1, 2, 4]] == 5) and torch.all(y[3] == ONE)
    santa.kv4_append(cache, x, x, ints([0] * B), workspace=ws)
    assert santa.device_status(ws) == 0


# ------------------------------------------------------------------ attention

def check(op, q, k, v, seq, window=0, sinks=0, scale=0.0, **kw):
    """One call against the reference; k, v CPU bf16 [B, H_kv, n, d] without NaN in use."""
    if op == "kv4":
        cache = filled_cache(k, v)
        kr, vr = held(cache)
        out = santa.decode_kv4(q.to(DEV), cache, ints(seq), window, sinks, scale, **kw)
    else:
        kr, vr = k.double().numpy(), v.double().numpy()
        out = santa.decode_window(q.to(DEV), k.to(DEV), v.to(DEV), ints(seq), window, sinks, scale, **kw)
    ref = kv4_util.attention(q, kr, vr, seq, window, sinks, scale)
    err = np.abs(out.cpu().double().numpy() - ref).max()
    assert err <= TOL * np.abs(np.nan_to_num(vr)).max(), err
    return out


def inputs(seed, seq, H_q, H_kv, d, n_max, std=3.0):
    g = gen(seed)
    q = workloads.make_q(len(seq), H_q, d, std, g)
    return q, rand(g, len(seq), H_kv, n_max, d), rand(g, len(seq), H_kv, n_max, d)


OPS = ["kv4", "window"]
SEQ = [1008, 1, 0, 2, 15, 16, 17, 31, 32, 33, 63, 65, 127, 129, 777]


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("d,H_q,H_kv", [(128, 32, 8), (128, 8, 8), (128, 8, 4), (128, 16, 2), (64, 4, 1), (64, 16, 2),
                                        (64, 3, 3), (64, 4, 2)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (16, 4), (100, 33), (500, 1), (2000, 5), (40, 2000)])
def test_attention(op, d, H_q, H_kv, window, sinks):
    q, k, v = inputs(d + H_q, SEQ, H_q, H_kv, d, 1008)
    out = check(op, q, k, v, SEQ, window, sinks)
    assert torch.all(out[2] == 0)


@pytest.mark.parametrize("op", OPS)
def test_unaligned_capacity_window_edges(op):
    """Every position of the window's start inside a tile, and odd capacities (bf16)."""
    n_max = 96 if op == "kv4" else 91
    for n in range(64, 91, 3):
        q, k, v = inputs(n, [n, n - 1], 4, 2, 64, n_max)
        check(op, q, k, v, [n, n - 1], n - 31, 3)
        check(op, q, k, v, [n, n - 1], 7, n - 20)


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("B,H_kv,n,window", [(1, 1, 20000, 0), (2, 2, 9000, 0), (40, 4, 700, 0), (3, 8, 5000, 4096),
                                             (200, 2, 150, 60)])
def test_attention_many_splits_and_many_rows(op, B, H_kv, n, window):
    n_max = -(-n // 16) * 16
    seq = [n - 7 * (b % 50) for b in range(B)]
    q, k, v = inputs(B + n, seq, 4 * H_kv, H_kv, 128, n_max)
    a = check(op, q, k, v, seq, window, 4)
    assert torch.equal(a, check(op, q, k, v, seq, window, 4))      # the same bits again


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("n", [511, 512, 513, 2047, 2048, 2049])
def test_where_groups_begin_to_be_split(op, n):
    """Few groups around the length up to which each has one CTA to itself, a short one and an
    empty one among them, and the same with more groups than SMs."""
    n_max = -(-n // 16) * 16
    q, k, v = inputs(n, [n, 5, 0], 8, 2, 128, n_max)
    check(op, q, k, v, [n, 5, 0])
    q, k, v = inputs(n, [n // 16] * 100, 4, 2, 64, 144)
    check(op, q, k, v, [min(n // 16 + b, 144) for b in range(100)])


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("n", [255, 256, 257, 1023, 1024, 1025])
def test_where_short_groups_begin_to_be_split(op, n):
    """Few groups around the length up to which each has one CTA to itself, a short one and an
    empty one among them, and the same with more groups than SMs."""
    n_max = -(-n // 16) * 16
    q, k, v = inputs(n, [n, 5, 0], 8, 2, 128, n_max)
    check(op, q, k, v, [n, 5, 0])
    q, k, v = inputs(n, [n // 16] * 100, 4, 2, 64, 144)
    check(op, q, k, v, [min(n // 16 + b, 144) for b in range(100)])


@pytest.mark.parametrize("op", OPS)
def test_many_batch_rows(op):
    """1024 batch rows (the most there may be), empty and short ones."""
    seq = [(7 * b) % 49 for b in range(1024)]
    q, k, v = inputs(1, seq, 2, 2, 64, 48)
    check(op, q, k, v, seq)
    check(op, q, k, v, seq, 16, 2)


@pytest.mark.parametrize("op", OPS)
def test_windows_and_sinks_beyond_the_cache(op):
    seq = [100, 33]
    q, k, v = inputs(2, seq, 4, 2, 64, 112)
    big = 2 ** 31 - 1
    every = check(op, q, k, v, seq)
    assert torch.equal(check(op, q, k, v, seq, big, big), every)
    assert torch.equal(check(op, q, k, v, seq, big, 0), every)
    check(op, q, k, v, seq, 7, big)


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("std,scale", [(0.0, 0.0), (0.1, 0.0), (3.0, 1e-3), (12.0, 0.0), (3.0, -0.1)])
def test_flat_and_peaked_scores_and_other_scales(op, std, scale):
    seq = [400, 1000]
    q, k, v = inputs(7, seq, 8, 2, 128, 1008, std)
    check(op, q, k, v, seq, 300, 10, scale)


@pytest.mark.parametrize("op", OPS)
def test_sizes_far_from_one(op):
    """Values of 1e-4 and of 1e4 (V), keys of 300 against queries of 1e-3, a query of 1e30."""
    seq = [600, 90]
    q, k, v = inputs(3, seq, 8, 2, 128, 608)
    check(op, q, k, (v.float() * 1e-4).bfloat16(), seq)
    check(op, q, k, (v.float() * 1e4).bfloat16(), seq)
    check(op, (q.float() * 1e-2).bfloat16(), (k.float() * 100).bfloat16(), v, seq)
    check(op, (q.float() * 1e30).bfloat16(), k, v, seq, scale=1e-31)


@pytest.mark.parametrize("op", OPS)
def test_bf16_output_is_the_fp32_result_rounded_once(op):
    seq = [500, 0, 33]
    q, k, v = inputs(11, seq, 16, 4, 128, 512)
    a = check(op, q, k, v, seq, 200, 4)
    buf = torch.empty(3, 16, 128, dtype=torch.bfloat16, device=DEV)
    if op == "kv4":
        b = santa.decode_kv4(q.to(DEV), filled_cache(k, v), ints(seq), 200, 4, out=buf)
    else:
        b = santa.decode_window(q.to(DEV), k.to(DEV), v.to(DEV), ints(seq), 200, 4, out=buf)
    assert b is buf and torch.equal(a.to(torch.bfloat16), b)


@pytest.mark.parametrize("op", OPS)
def test_keys_that_are_not_visible_do_not_matter(op):
    """NaN and infinities in every masked place (behind the sequence, before the window), and
    in the rows of an empty sequence."""
    seq, window, sinks = [300, 77, 0, 16], 45, 3
    q, k, v = inputs(5, seq, 8, 2, 64, 320)
    clean = check(op, q, k, v, seq, window, sinks)
    for b, n in enumerate(seq):
        hide = np.setdiff1d(np.arange(320), kv4_util.visible(n, window, sinks))
        k[b][:, hide[0::2]], v[b][:, hide[0::2]] = NAN, float("inf")
        k[b][:, hide[1::2]], v[b][:, hide[1::2]] = float("-inf"), NAN
    if op == "kv4":
        out = santa.decode_kv4(q.to(DEV), filled_cache(k, v), ints(seq), window, sinks)
    else:
        out = santa.decode_window(q.to(DEV), k.to(DEV), v.to(DEV), ints(seq), window, sinks)
    assert torch.equal(out, clean)


@pytest.mark.parametrize("op", OPS)
def test_nan_in_a_visible_place_shows(op):
    """A NaN among the visible values shows in its batch row and KV head and nowhere else."""
    seq = [100, 100]
    q, k, v = inputs(6, seq, 8, 2, 64, 112)
    clean = check(op, q, k, v, seq)
    k[0, 1, 37, 5] = NAN
    v[1, 0, 99, 20] = NAN
    if op == "kv4":
        out = santa.decode_kv4(q.to(DEV), filled_cache(k, v), ints(seq))
    else:
        out = santa.decode_window(q.to(DEV), k.to(DEV), v.to(DEV), ints(seq), 0)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[0, 4:] = True
    bad[1, :4, 16:32] = True if op == "kv4" else bad[1, :4, 16:32]
    bad[1, :4, 20] = True
    assert torch.equal(torch.isnan(out), bad)
    assert torch.equal(out[~bad], clean[~bad])


@pytest.mark.parametrize("op", OPS)
def test_bad_lengths_are_reported_and_give_zeros(op):
    q, k, v = inputs(9, [64, 64, 64], 4, 2, 64, 64)
    ws = santa.new_workspace(santa.workspace_size(santa.make_shape(3, 4, 2, 64, 64), 16, "systematic") + (8 << 20), DEV)
    sl = ints([65, 64, -1])
    if op == "kv4":
        call = lambda: santa.decode_kv4(q.to(DEV), filled_cache(k, v), sl, 9, 1, workspace=ws)  # noqa: E731
    else:
        call = lambda: santa.decode_window(q.to(DEV), k.to(DEV), v.to(DEV), sl, 9, 1, workspace=ws)  # noqa: E731
    out = call()
    assert santa.device_status(ws) == santa.DEV_BAD_SEQLEN and santa.device_status(ws) == 0
    assert torch.all(out[0] == 0) and torch.all(out[2] == 0) and out[1].abs().max() > 0


def test_offsets_past_32_bits():
    """Caches whose last rows start past 2^32 bytes; only those rows are read or written."""
    d, H_kv = 128, 8
    B, n_max = 17, 524288                                   # 71M rows of 64 bytes: 4.6 GB a tensor
    cache = santa.KV4Cache(*(torch.empty(B, H_kv, n_max, w, dtype=torch.uint8, device=DEV) for w in (64, 8, 64, 8)))
    assert cache.k.numel() > 1 << 32
    g = gen(1)
    T, seq = 300, [0] * (B - 1) + [n_max]
    k, v = rand(g, 1, T, H_kv, d), rand(g, 1, T, H_kv, d)
    full = torch.zeros(B, T, H_kv, d, dtype=torch.bfloat16, device=DEV)
    counts = ints([0] * (B - 1) + [T])
    pos = ints([0] * (B - 1) + [n_max - T])
    kn, vn = full.clone(), full
    kn[-1], vn[-1] = k[0].to(DEV), v[0].to(DEV)
    santa.kv4_append(cache, kn, vn, pos, counts)
    ko, vo = torch.zeros_like(kn), torch.zeros_like(vn)
    santa.kv4_read(cache, pos, ko, vo, counts)
    ck, cv = (kv4_util.values(*kv4_util.quantise(x[0].transpose(0, 1).contiguous())) for x in (k, v))
    assert np.array_equal(ko[-1].transpose(0, 1).cpu().double().numpy(), ck)
    assert np.array_equal(vo[-1].transpose(0, 1).cpu().double().numpy(), cv)
    q = workloads.make_q(B, 16, d, 3.0, g)
    out = santa.decode_kv4(q.to(DEV), cache, ints(seq), window=T)
    ref = kv4_util.attention(q[-1:], ck[None], cv[None], [T])
    assert np.abs(out[-1:].cpu().double().numpy() - ref).max() <= TOL * np.abs(cv).max()
    assert torch.all(out[:-1] == 0)
    del cache, kn, vn, ko, vo, full
    torch.cuda.empty_cache()
    B, n_max = 3, 400000                                    # 9.6M rows of 256 bytes: 2.5 GB of bf16 elements x 2
    kc, vc = (torch.empty(B, H_kv, n_max, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    kc[-1, :, -T:], vc[-1, :, -T:] = k[0].transpose(0, 1).to(DEV), v[0].transpose(0, 1).to(DEV)
    out = santa.decode_window(q[:B].to(DEV), kc, vc, ints([0, 0, n_max]), T)
    ref = kv4_util.attention(q[B - 1:B], k.transpose(1, 2), v.transpose(1, 2), [T])
    assert np.abs(out[-1:].cpu().double().numpy() - ref).max() <= TOL * float(v.abs().max())


# ------------------------------------------------------------------ use

def test_workspace_shared_with_sampled_and_dense_decodes():
    """One workspace for every kind of call, in any order: results are those of a fresh one."""
    seq = [3000, 777, 0, 2049]
    q, k, v = (x.to(DEV) for x in inputs(21, seq, 16, 4, 128, 3008))
    sl, cache = ints(seq), filled_cache(k.cpu(), v.cpu())
    n = max(santa.workspace_size(santa.make_shape(4, 16, 4, 128, 3008), 96, m) for m in ("systematic", "dense"))
    ws = santa.new_workspace(n + (16 << 20), DEV)
    small = ints([50, 1])
    calls = [lambda w: santa.decode(q, k, v, sl, 96, "systematic", seed=5, workspace=w, two_pass=True)[0],
             lambda w: santa.decode_window(q, k, v, sl, 500, 4, workspace=w),
             lambda w: santa.decode(q, k, v, sl, 1, "dense", workspace=w)[0],
             lambda w: santa.decode_kv4(q, cache, sl, workspace=w),
             lambda w: santa.decode_window(q[:2], k[:2], v[:2], small, 9, 2, workspace=w)]
    want = [c(None).clone() for c in calls]
    for order in ([0, 1, 2, 3, 4], [3, 0, 4, 1, 2], [1, 3, 1, 0, 3]):
        for i in order:
            assert torch.equal(calls[i](ws), want[i]), i
    assert santa.device_status(ws) == 0


def test_streams_at_once():
    """Calls on two streams at the same time, each with its own workspace."""
    seq = [4000] * 4
    q, k, v = (x.to(DEV) for x in inputs(2, seq, 32, 8, 128, 4000))
    sl, cache = ints(seq), filled_cache(k.cpu(), v.cpu())
    want = [santa.decode_kv4(q, cache, sl), santa.decode_window(q, k, v, sl, 2500, 4)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(santa.decode_kv4(q, cache, sl) if i == 0 else santa.decode_window(q, k, v, sl, 2500, 4))
    explicit = santa.decode_window(q, k, v, sl, 2500, 4, stream=streams[0])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])
    assert torch.equal(explicit, want[1])


def _reference_steps(k0, v0, counts, steps, q, window, sinks):
    """Quantised prompt, then per step one more token and the attention over all of them."""
    quant = lambda x: kv4_util.values(*kv4_util.quantise(x))  # noqa: E731
    B = len(counts)
    ks = [quant(k0[b, :counts[b]].transpose(0, 1).contiguous()) for b in range(B)]
    vs = [quant(v0[b, :counts[b]].transpose(0, 1).contiguous()) for b in range(B)]
    outs = []
    for t, (kn, vn) in enumerate(steps):
        out = []
        for b in range(B):
            ks[b] = np.concatenate([ks[b], quant(kn[b].transpose(0, 1).contiguous())], 1)
            vs[b] = np.concatenate([vs[b], quant(vn[b].transpose(0, 1).contiguous())], 1)
            out.append(kv4_util.attention(q[t][b:b + 1], ks[b][None], vs[b][None], [ks[b].shape[1]], window, sinks)[0])
        outs.append(np.stack(out))
    return outs


@pytest.mark.parametrize("captured", [False, True])
def test_prompt_then_decode_steps(captured):
    """A ragged padded prompt, then decode steps of append, length update and attention under
    a window that the generation outgrows; eager, and as one captured step replayed with new
    inputs in the same buffers while a second captured graph runs on another stream."""
    g = gen(17)
    B, T, H_q, H_kv, d, n_max, window, sinks, n_steps = 3, 40, 8, 2, 128, 96, 24, 4, 12
    counts = [40, 9, 23]
    k0, v0 = rand(g, B, T, H_kv, d), rand(g, B, T, H_kv, d)
    steps = [(rand(g, B, 1, H_kv, d), rand(g, B, 1, H_kv, d)) for _ in range(n_steps)]
    q = [workloads.make_q(B, H_q, d, 3.0, g) for _ in range(n_steps)]
    want = _reference_steps(k0, v0, counts, steps, q, window, sinks)
    cache = santa.new_kv4_cache(B, H_kv, n_max, d)
    santa.kv4_append(cache, k0.to(DEV), v0.to(DEV), ints([0] * B), ints(counts))
    lens = ints(counts)
    qb = torch.zeros(B, H_q, d, dtype=torch.bfloat16, device=DEV)
    kb, vb = (torch.zeros(B, 1, H_kv, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    out = torch.zeros(B, H_q, d, device=DEV)

    def step():
        santa.kv4_append(cache, kb, vb, lens)
        lens.add_(1)
        santa.decode_kv4(qb, cache, lens, window, sinks, out=out)

    graph = other = None
    if captured:
        start = lens.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        assert torch.equal(lens, start)                      # capturing ran nothing
        oq, ok, ov = (x.to(DEV) for x in inputs(4, [700], 8, 2, 128, 700))
        osl, oout = ints([700]), torch.zeros(1, 8, 128, device=DEV)
        owant = santa.decode_window(oq, ok, ov, osl, 600, 3)
        other = torch.cuda.CUDAGraph()
        with torch.cuda.graph(other):
            santa.decode_window(oq, ok, ov, osl, 600, 3, out=oout)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
    for t in range(n_steps):
        qb.copy_(q[t]), kb.copy_(steps[t][0]), vb.copy_(steps[t][1])
        if captured:
            with torch.cuda.stream(side):
                other.replay()
            graph.replay()
        else:
            step()
        torch.cuda.synchronize()
        assert np.abs(out.cpu().double().numpy() - want[t]).max() <= TOL * 6
        if captured:
            assert torch.equal(oout, owant)
            oout.zero_()


def test_reading_back_feeds_the_sampled_modes():
    """The 4-bit cache read into a bf16 cache: sampling there (every S-th point of a flat
    softmax) and the exact step agree with decode_kv4 on the same values."""
    seq = [2000, 333]
    q, k, v = inputs(8, seq, 8, 2, 128, 2000)
    cache = filled_cache(k, v)
    kb, vb = (torch.zeros(2, 2, 2000, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    santa.kv4_read(cache, ints([0, 0]), kb.transpose(1, 2), vb.transpose(1, 2), ints(seq))
    a = santa.decode_kv4(q.to(DEV), cache, ints(seq))
    b, _ = santa.decode(q.to(DEV), kb, vb, ints(seq), 1, "dense")
    c = santa.decode_window(q.to(DEV), kb, vb, ints(seq), 0)
    big = float(vb.abs().max())
    assert (a - b).abs().max() <= 2 * TOL * big and (a - c).abs().max() <= 2 * TOL * big
    est, idx = santa.decode(q.to(DEV), kb, vb, ints(seq), 4096, "systematic", seed=1)
    assert int(idx[1].max()) < 333
    # 4096 systematic points: each key's share is off by less than one point
    assert (est - a).norm() / a.norm() < 0.1


def test_binding_refuses_mismatched_tensors():
    z = torch.zeros
    cache = santa.new_kv4_cache(2, 2, 32, 64)
    x, pos = z(2, 3, 2, 64, dtype=torch.bfloat16, device=DEV), ints([0, 0])
    bad = [(x.float(), x, pos, None), (x[:1], x[:1], pos, None), (x, x[:, :2], pos, None), (x[..., :32], x, pos, None),
           (x, x.transpose(2, 3).contiguous().transpose(2, 3), pos, None), (x, x.cpu(), pos, None),
           (x, x, pos.long(), None), (x, x, pos[:1], None), (x, x, pos, pos.float()), (x, x, pos.cpu(), None)]
    for k, v, p, c in bad:
        with pytest.raises(ValueError):
            santa.kv4_append(cache, k, v, p, c)
    with pytest.raises(ValueError):
        santa.kv4_append(cache._replace(v=cache.v[:, :1]), x, x, pos)
    with pytest.raises(ValueError):
        santa.kv4_append(cache._replace(k=cache.k.transpose(0, 1)), x, x, pos)
    q = z(2, 4, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        santa.decode_kv4(q.float(), cache, pos)
    with pytest.raises(ValueError):
        santa.decode_kv4(q[:1], cache, pos)
    with pytest.raises(ValueError):
        santa.decode_kv4(q, cache, pos.long())
    with pytest.raises(ValueError):
        santa.decode_kv4(q, cache, pos, out=z(2, 4, 64, dtype=torch.float16, device=DEV))
    with pytest.raises(santa.SantaError):
        santa.decode_kv4(q, cache, pos, window=-1)
    kc = z(2, 2, 30, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        santa.decode_window(q, kc, kc[:, :, :20], pos, 4)
    with pytest.raises(ValueError):
        santa.decode_window(q, kc.transpose(1, 2), kc, pos, 4)
    with pytest.raises(ValueError):
        santa.decode_kv4(q, cache, pos, window=1 << 31)
    with pytest.raises(ValueError):                 # K and V read into the same rows
        santa.kv4_read(cache, pos, x, x)
    with pytest.raises(santa.SantaError) as e:      # queries that begin between two 16-byte boundaries
        room = z(2 * 4 * 64 + 8, dtype=torch.bfloat16, device=DEV)
        santa.decode_kv4(room[4:4 + 512].view(2, 4, 64), cache, pos)
    assert e.value.status == -2
    with pytest.raises(santa.SantaError) as e:
        santa.decode_kv4(q, cache, pos, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    assert e.value.status == -3
