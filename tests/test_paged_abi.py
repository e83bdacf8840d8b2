"""The entry points of rotary positions and of the paged cache, without a GPU: refusals come from
the host, before anything is enqueued (the addresses and the stream are made up), the binding checks
its tensors, and the table of frequencies agrees with its formulas."""
import ctypes
import math

import numpy as np
import pytest
import torch

from stochastic_sparse_kv_gb300 import santa, _build
from tests import paged_util

A = 1 << 20          # a made-up, aligned address
STREAM = 0xDEAD0     # a made-up stream
i64 = ctypes.c_int64 * 3


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return santa.load()


def shape(B=2, H_q=8, H_kv=2, d=128, n_max=256, scale=0.0):
    return ctypes.byref(santa.make_shape(B, H_q, H_kv, d, n_max, scale))


def pool(k=A, v=2 * A, table=A, n_pages=40, page=16):
    return ctypes.byref(santa._Paged(k, v, table, n_pages, page))


def rows(k=A, v=A, ks=(4096, 256, 128), vs=(4096, 256, 128)):
    return ctypes.byref(santa._Rows(k, v, ks, vs))


def rot(turns=A, rot=128, layout=0, amplitude=1.0):
    return ctypes.byref(santa._Rotation(turns, rot, layout, amplitude))


def test_rope_refusals(lib):
    def call(B=2, T=4, H=2, d=128, x=A, xs=(4096, 256, 128), out=A, os=(4096, 256, 128), r=None, pos=A, counts=None, ws=None):
        return lib.santa_rope(B, T, H, d, x, i64(*xs) if xs else None, out, i64(*os) if os else None, r or rot(), pos,
                              counts, ws, STREAM)

    assert call(T=0) == 0                                    # nothing to do: nothing enqueued
    assert call(B=0) == -1 and call(T=-1) == -1 and call(H=0) == -1 and call(d=0) == -1
    assert call(x=None) == -1 and call(out=None) == -1 and call(pos=None) == -1 and call(xs=None) == -1 and call(os=None) == -1
    assert call(d=96) == -4 and call(B=1025) == -4 and call(H=1025) == -4
    assert call(x=A + 8) == -2 and call(out=A + 2) == -2 and call(pos=A + 2) == -2 and call(counts=A + 1) == -2
    assert call(ws=A + 16) == -2
    assert call(xs=(4096, 260, 128)) == -2 and call(xs=(4096, -256, 128)) == -1
    assert call(os=(4096, 256, 0)) == -1 and call(os=(0, 256, 128)) == -1 and call(os=(4096, 128, 128)) == -1
    assert call(r=rot(turns=None)) == -1 and call(r=rot(turns=A + 4)) == -2 and call(r=rot(layout=2)) == -1
    assert call(r=rot(amplitude=math.nan)) == -1 and call(r=rot(amplitude=math.inf)) == -1
    for bad in (0, 8, 24, 144, -16):
        assert call(r=rot(rot=bad)) == -4
    assert call(d=64, r=rot(rot=80), xs=(4096, 256, 64), os=(4096, 256, 64)) == -4
    assert call(B=1024, H=1024, T=1 << 20, xs=(0, 0, 0), os=(1 << 40, 1 << 20, 128)) == -4   # too many rows
    assert lib.santa_rope(2, 4, 2, 128, A, i64(4096, 256, 128), A, i64(4096, 256, 128), None, A, None, None, STREAM) == -1


def test_append_refusals(lib):
    def call(sh=None, c=None, r=None, T=4, pos=A, counts=None, ro=None, q=None, qs=None, qo=None, qos=None, ws=None):
        return lib.santa_paged_append(sh or shape(), c or pool(), r or rows(), T, pos, counts, ro, q, i64(*qs) if qs else None,
                                      qo, i64(*qos) if qos else None, ws, STREAM)

    st = (4096, 1024, 128)
    assert call(T=0) == 0 and call(T=0, ro=rot(), q=A, qs=st, qo=A, qos=st) == 0
    assert call(T=-1) == -1 and call(pos=None) == -1 and call(r=rows(k=None)) == -1 and call(r=rows(v=None)) == -1
    assert call(c=pool(k=None)) == -1 and call(c=pool(v=None)) == -1 and call(c=pool(table=None)) == -1
    assert call(c=pool(n_pages=0)) == -1 and call(c=pool(v=A)) == -1                 # one pool for K and V
    for page in (0, 8, 24, 48, 512, -16):
        assert call(c=pool(page=page)) == -4
    assert call(sh=shape(n_max=100)) == -4 and call(sh=shape(n_max=524288 + 16)) == -4 and call(sh=shape(n_max=0)) == -1
    assert call(c=pool(n_pages=1 << 26)) == -4               # pool rows beyond 2^31
    assert call(sh=shape(d=96)) == -4 and call(sh=shape(B=0)) == -1 and call(sh=shape(B=1025)) == -4
    assert call(c=pool(k=A + 8)) == -2 and call(c=pool(table=A + 2)) == -2 and call(r=rows(k=A + 2)) == -2
    assert call(pos=A + 2) == -2 and call(counts=A + 1) == -2 and call(ws=A + 16) == -2
    assert call(r=rows(ks=(4096, 260, 128))) == -2 and call(r=rows(vs=(-4096, 256, 128))) == -1
    assert call(ro=rot(rot=24)) == -4 and call(ro=rot(layout=-1)) == -1
    assert call(ro=rot(), q=A, qs=st) == -1 and call(ro=rot(), qo=A, qos=st) == -1   # one without the other
    assert call(q=A, qs=st, qo=A, qos=st) == -1                                      # queries, but no rotation
    assert call(ro=rot(), q=A, qs=None, qo=A, qos=st) == -1
    assert call(ro=rot(), q=A + 8, qs=st, qo=A, qos=st) == -2
    assert call(ro=rot(), q=A, qs=st, qo=A, qos=(4096, 128, 128)) == -1              # rows that share memory
    assert call(sh=shape(B=1024, H_q=64, H_kv=64), c=pool(n_pages=1), T=1 << 20) == -4
    assert lib.santa_paged_append(None, pool(), rows(), 4, A, None, None, None, None, None, None, None, STREAM) == -1
    assert lib.santa_paged_append(shape(), None, rows(), 4, A, None, None, None, None, None, None, None, STREAM) == -1
    assert lib.santa_paged_append(shape(), pool(), None, 4, A, None, None, None, None, None, None, None, STREAM) == -1


def test_attend_refusals(lib):
    n = ctypes.c_size_t(0)
    assert lib.santa_attend_workspace_size(shape(), 4, ctypes.byref(n)) == 0
    assert n.value >= 65536 and n.value % 256 == 0

    def call(sh=None, q=A, qs=(4096, 1024, 128), c=None, T=4, pos=A, counts=None, window=16, sinks=2, out=A, ws=A, wsn=n.value):
        return lib.santa_attend_paged(sh or shape(), q, i64(*qs) if qs else None, c or pool(), T, pos, counts, window, sinks,
                                      out, ws, wsn, STREAM)

    assert call(T=0) == 0
    assert call(q=None) == -1 and call(qs=None) == -1 and call(pos=None) == -1 and call(out=None) == -1
    assert call(T=-1) == -1 and call(window=-1) == -1 and call(sinks=-1) == -1
    assert call(T=524289) == -4
    assert call(ws=None) == -3 and call(wsn=n.value - 1) == -3 and call(ws=A + 64) == -2
    assert call(q=A + 8) == -2 and call(out=A + 4) == -2 and call(pos=A + 2) == -2 and call(counts=A + 2) == -2
    assert call(qs=(4096, 1028, 128)) == -2 and call(qs=(4096, 1024, -128)) == -1
    assert call(sh=shape(H_q=9)) == -1 and call(sh=shape(H_q=32)) == -4 and call(sh=shape(d=32)) == -4
    assert call(sh=shape(scale=math.nan)) == -1 and call(sh=shape(scale=-0.5)) == -1 and call(sh=shape(scale=3e38)) == -1
    assert call(c=pool(v=None)) == -1 and call(c=pool(v=A + 8)) == -2 and call(sh=shape(n_max=40)) == -4
    assert call(c=pool(page=8)) == -4
    assert lib.santa_attend_paged(shape(), A, i64(0, 0, 0), None, 4, A, None, 0, 0, A, A, n.value, STREAM) == -1
    assert lib.santa_attend_workspace_size(shape(), 4, None) == -1 and lib.santa_attend_workspace_size(None, 4, ctypes.byref(n)) == -1
    assert lib.santa_attend_workspace_size(shape(), -1, ctypes.byref(n)) == -1
    assert lib.santa_attend_workspace_size(shape(B=1025), 4, ctypes.byref(n)) == -4
    # the batch's keys together are not limited, one sequence's are
    assert lib.santa_attend_workspace_size(shape(B=1024, n_max=524288), 4, ctypes.byref(n)) == 0


def test_turns_refusals(lib):
    def call(rot=64, base=10000.0, scaling=0, factor=2.0, low=1.0, high=4.0, original=8192, turns=True, amp=True, spec=True):
        s = santa._RopeSpec(base, scaling, factor, low, high, original)
        t, a = (ctypes.c_uint64 * 64)(), ctypes.c_float(0)
        return lib.santa_rope_turns(ctypes.byref(s) if spec else None, rot, t if turns else None, ctypes.byref(a) if amp else None)

    for how in range(5):
        assert call(scaling=how) == 0
    assert call(scaling=5) == -1 and call(scaling=-1) == -1
    assert call(rot=0) == -1 and call(rot=7) == -1 and call(rot=-2) == -1
    assert call(base=1.0) == -1 and call(base=math.inf) == -1 and call(base=math.nan) == -1
    assert call(scaling=1, factor=0.5) == -1 and call(scaling=1, factor=math.nan) == -1 and call(scaling=0, factor=0.0) == 0
    assert call(scaling=3, low=0.0) == -1 and call(scaling=3, low=4.0) == -1 and call(scaling=4, high=math.inf) == -1
    assert call(scaling=4, original=0) == -1 and call(scaling=2, original=0) == 0
    assert call(turns=False) == -1 and call(amp=False) == -1 and call(spec=False) == -1


@pytest.mark.parametrize("scaling", list(santa.ROPE_SCALINGS))
@pytest.mark.parametrize("rot", [16, 48, 128])
@pytest.mark.parametrize("base,factor,original", [(10000.0, 1.0, 2048), (500000.0, 8.0, 8192), (1e6, 32.5, 4096)])
def test_frequencies(lib, scaling, rot, base, factor, original):
    """To a step of the fixed point (2^-64 turns) and a few of a double."""
    t = santa.rope_table(rot, base, scaling=scaling, factor=factor, original=original, device="cpu")
    f, amplitude = paged_util.frequencies(rot, base, scaling, factor, original=original)
    turns = t.turns.numpy().view(np.uint64).astype(np.float64) * 2.0 ** -64
    assert np.abs(turns - f / (2 * math.pi)).max() <= 2.0 ** -64 + 2.0 ** -46
    assert np.abs(turns * 2 * math.pi / f - 1).max() <= 1e-10
    assert abs(t.amplitude - amplitude) <= 2.0 ** -24 * amplitude
    assert turns[0] * 2 * math.pi == pytest.approx(f[0], rel=1e-14) and (np.diff(turns) < 0).all()


def test_binding_checks_tensors():
    z = torch.zeros
    bf = torch.bfloat16
    cache = santa.new_paged_cache(4, 2, 16, 64, 1, 3, device="cpu")
    assert cache.k.shape == (4, 2, 16, 64) and cache.table.tolist() == [[-1, -1, -1]]
    table = santa.rope_table(64, device="cpu")
    x, pos = z(1, 3, 2, 64, dtype=bf), z(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        santa.rope(x, table, pos)
    with pytest.raises(ValueError, match="CUDA"):
        santa.paged_append(cache, x, x, pos)
    with pytest.raises(ValueError, match="CUDA"):
        santa.attend_paged(x, cache, pos)
    with pytest.raises(ValueError, match="layout"):
        santa.rope_table(64, layout="quarters")
    with pytest.raises(ValueError, match="scaling"):
        santa.rope_table(64, scaling="more")
    with pytest.raises(santa.SantaError):
        santa.rope_table(64, base=0.5)


def test_reference_on_known_values():
    """The reference itself: one pair a quarter turn on, and attention that averages two keys."""
    x = torch.zeros(1, 1, 1, 64).bfloat16()
    x[..., 0], x[..., 1], x[..., 32] = 2.0, 3.0, 5.0
    f = np.zeros(32)
    f[0] = math.pi / 2
    assert np.allclose(paged_util.rotate(x, f, 1.0, "halves", [1])[0, 0, 0, [0, 1, 32]], [-5, 3, 2])
    assert np.allclose(paged_util.rotate(x, f, 1.0, "pairs", [1])[0, 0, 0, [0, 1, 32]], [-3, 2, 5])
    k, v = torch.zeros(2, 1, 16, 64), torch.zeros(2, 1, 16, 64)
    v[1, 0, 0], v[1, 0, 1] = 1, 3
    o, spread = paged_util.attention(torch.zeros(1, 2, 1, 64), k, v, torch.tensor([[1]]), [0])
    assert np.allclose(o[0, 0], 1) and np.allclose(o[0, 1], 2) and np.allclose(spread[0, 1], 1)
