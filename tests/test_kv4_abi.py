"""The entry points of the 4-bit cache and of windowed attention, without a GPU: refusals come
from the host, before anything is enqueued (the addresses and the stream are made up), and the
binding checks its tensors.  Also the 64-bit reference of the format against facts."""
import ctypes

import numpy as np
import pytest
import torch

from stochastic_sparse_kv_gb300 import santa, _build
from tests import kv4_util

A = 1 << 20          # a made-up, aligned address
STREAM = 0xDEAD0     # a made-up stream


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return santa.load()


def shape(B=2, H_q=8, H_kv=2, d=128, n_max=64, scale=0.0):
    return ctypes.byref(santa.make_shape(B, H_q, H_kv, d, n_max, scale))


def rows(k=A, v=A, ks=(4096, 256, 128), vs=(4096, 256, 128)):
    return ctypes.byref(santa._Rows(k, v, ks, vs))


def kv(k=A, ks=A, v=A, vs=A):
    return ctypes.byref(santa._Kv4(k, ks, v, vs))


@pytest.mark.parametrize("name", ["santa_kv4_append", "santa_kv4_read"])
def test_move_refusals(lib, name):
    def call(sh=None, c=None, r=None, T=4, pos=A, counts=None, ws=None):
        return getattr(lib, name)(sh or shape(), c or kv(), r or rows(), T, pos, counts, ws, STREAM)

    assert call(T=0) == 0                                   # nothing to do: nothing enqueued
    assert call(T=-1) == -1
    assert call(pos=None) == -1
    assert call(c=kv(k=None)) == -1 and call(c=kv(vs=None)) == -1
    assert call(r=rows(v=None)) == -1
    assert call(sh=shape(n_max=72)) == -4                   # capacity not a multiple of 16
    assert call(sh=shape(d=96)) == -4
    assert call(sh=shape(B=0)) == -1
    assert call(c=kv(ks=A + 8)) == -2 and call(r=rows(k=A + 2)) == -2
    assert call(pos=A + 2) == -2 and call(counts=A + 1) == -2 and call(ws=A + 16) == -2
    assert call(r=rows(ks=(4096, 260, 128))) == -2          # stride not a multiple of 8
    assert call(r=rows(vs=(-4096, 256, 128))) == -1
    assert call(sh=shape(B=1024, H_q=16, H_kv=16, n_max=16384), T=1 << 20) == -4   # too many groups
    assert lib.santa_kv4_append(None, kv(), rows(), 4, A, None, None, STREAM) == -1
    assert lib.santa_kv4_append(shape(), None, rows(), 4, A, None, None, STREAM) == -1
    assert lib.santa_kv4_append(shape(), kv(), None, 4, A, None, None, STREAM) == -1


def test_read_refuses_rows_that_share_memory(lib):
    def call(st, T=4, **kw):
        return lib.santa_kv4_read(shape(**kw), kv(), rows(ks=st), T, A, None, None, STREAM)

    assert call((4096, 256, 0)) == -1          # one row for all heads
    assert call((0, 256, 128)) == -1           # one row for all batch rows
    assert call((256, 256, 128)) == -1         # batch rows inside one another's tokens
    assert call((4096, 128, 128)) == -1        # tokens inside one another's heads
    assert call((4096, 128, 384)) == -1        # head-major, heads closer than 4 tokens
    # tokens 2^39 apart reach past 2^63, batch rows 2^40 apart lie among them
    far = (1 << 40, 1 << 39, 64)
    assert lib.santa_kv4_read(shape(B=2, H_q=1, H_kv=1, d=64), kv(), rows(ks=far, vs=far), (1 << 28) - 1, A, None, None, STREAM) == -1
    # strides of dimensions of size 1 (or 0) are not read; nothing to do, so nothing is enqueued
    # (one row with such strides is read in test_kv4_gpu.py)
    assert call((-3, 1, 7), T=0, B=1, H_kv=1) == 0


@pytest.mark.parametrize("name", ["santa_decode_kv4", "santa_decode_window"])
def test_decode_refusals(lib, name):
    n = ctypes.c_size_t(0)
    assert lib.santa_window_workspace_size(shape(), ctypes.byref(n)) == 0
    assert n.value >= 65536 and n.value % 256 == 0

    def call(sh=None, q=A, c=None, k=A, v=A, sl=A, window=16, sinks=2, flags=0, out=A, ws=A, wsn=n.value):
        cache = (c or kv(),) if name == "santa_decode_kv4" else (k, v)
        return getattr(lib, name)(sh or shape(), q, *cache, sl, window, sinks, flags, out, ws, wsn, STREAM)

    assert call(q=None) == -1 and call(sl=None) == -1 and call(out=None) == -1
    assert call(window=-1) == -1 and call(sinks=-1) == -1
    assert call(flags=santa.OUT_BF16 | santa.GROUP_DEDUP) == -1 and call(flags=1) == -1
    assert call(ws=None) == -3 and call(wsn=n.value - 1) == -3
    assert call(q=A + 8) == -2 and call(out=A + 4) == -2 and call(sl=A + 2) == -2 and call(ws=A + 64) == -2
    assert call(sh=shape(H_q=9)) == -1 and call(sh=shape(H_q=32)) == -4 and call(sh=shape(d=32)) == -4
    assert call(sh=shape(scale=float("nan"))) == -1
    if name == "santa_decode_kv4":
        assert call(c=kv(v=None)) == -1 and call(c=kv(v=A + 8)) == -2 and call(sh=shape(n_max=40)) == -4
    else:
        assert call(k=None) == -1 and call(v=A + 8) == -2
    assert lib.santa_window_workspace_size(shape(), None) == -1
    assert lib.santa_window_workspace_size(None, ctypes.byref(n)) == -1
    # more (batch row, KV head) groups than the control block has counters
    assert lib.santa_window_workspace_size(shape(B=1024, H_q=32, H_kv=16, n_max=16), ctypes.byref(n)) == -4


def test_binding_checks_tensors():
    z = torch.zeros
    cache = santa.KV4Cache(z(1, 2, 32, 32, dtype=torch.uint8), z(1, 2, 32, 4, dtype=torch.uint8),
                           z(1, 2, 32, 32, dtype=torch.uint8), z(1, 2, 32, 4, dtype=torch.uint8))
    q, pos = z(1, 4, 64, dtype=torch.bfloat16), z(1, dtype=torch.int32)
    rows_ = z(1, 3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        santa.kv4_append(cache, rows_, rows_, pos)
    with pytest.raises(ValueError, match="CUDA"):
        santa.kv4_read(cache, pos, rows_, rows_)
    with pytest.raises(ValueError, match="CUDA"):
        santa.decode_kv4(q, cache, pos)
    with pytest.raises(ValueError, match="CUDA"):
        santa.decode_window(q, z(1, 2, 32, 64, dtype=torch.bfloat16), z(1, 2, 32, 64, dtype=torch.bfloat16), pos, 8)
    new = santa.new_kv4_cache(2, 3, 17, 64, device="cpu")
    assert new.k.shape == (2, 3, 32, 32) and new.v_scale.shape == (2, 3, 32, 4)


def test_reference_scale_is_fp16_bits():
    codes = np.arange(0xF8, dtype=np.uint16)
    assert np.array_equal((codes << 7).view(np.float16).astype(np.float64), kv4_util.SCALE[:0xF8])
    assert np.isnan(kv4_util.SCALE[0xF8:]).all() and kv4_util.SCALE[kv4_util.MAX_CODE] == 10240


def test_reference_quantiser_on_known_groups():
    x = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, 0.0])
    c, s = kv4_util.quantise(x.to(torch.bfloat16))
    assert s[0] == 15 << 3                                             # scale 1
    want = [6, 0, 1, 1, 2, 2, 4, 4, 0, -1, -1, -2, -2, -4, -4, 0]      # ties to the even index
    assert kv4_util.values(c, s).tolist() == want
    assert kv4_util.values(*kv4_util.quantise(torch.full((16,), 3e38).to(torch.bfloat16))).tolist() == [61440.0] * 16
    assert np.isnan(kv4_util.values(*kv4_util.quantise(torch.tensor([float("inf")] + [1.0] * 15).bfloat16()))).all()
