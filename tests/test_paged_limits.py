"""Limits of the calls over a paged cache that a number in C could hide, without a GPU: the flag in T and
numbers past 32 bits."""
import ctypes

import pytest

from stochastic_sparse_kv_gb300 import santa
from tests.test_paged_abi import A, STREAM, i64, lib, pool, rot, rows, shape  # noqa: F401  (lib: fixture)


def test_the_flag_in_T_changes_no_check(lib):  # noqa: F811
    n = ctypes.c_size_t(0)
    assert lib.santa_attend_workspace_size(shape(), 4, ctypes.byref(n)) == 0
    st = (1 << 38, 1024, 128)
    for clear in (0, santa.CLEAR_REST):
        rope = lambda T, **k: lib.santa_rope(k.get("B", 2), T | clear, 2, 128, A, i64(*st), A, i64(*st), rot(), A, None, None, STREAM)  # noqa: E731
        append = lambda T, **k: lib.santa_paged_append(k.get("sh", shape()), pool(), rows(), T | clear, A, None, rot(), A, i64(*st), A,  # noqa: E731
                                                       i64(*st), None, STREAM)
        attend = lambda T, ws=A: lib.santa_attend_paged(shape(), A, i64(*st), pool(), T | clear, A, None, 0, 0, A, ws, n.value, STREAM)  # noqa: E731
        assert rope(0) == append(0) == attend(0) == 0
        assert rope(1 << 27) == -4 and append(1 << 27) == -4
        assert attend(524289) == -4 and attend(5) == -3 and attend(4, ws=None) == -3
        assert rope(4, B=0) == -1 and append(4, sh=shape(B=0)) == -1
    for T in (-1, -(1 << 31)):
        assert lib.santa_rope(2, T, 2, 128, A, i64(*st), A, i64(*st), rot(), A, None, None, STREAM) == -1
        assert lib.santa_attend_paged(shape(), A, i64(*st), pool(), T, A, None, 0, 0, A, A, n.value, STREAM) == -1


def test_numbers_past_32_bits_of_a_rope_table(lib):  # noqa: F811
    """(a C argument takes the low 32 bits: 2^32 + 8192 positions were 8192)"""
    for bad in (dict(original=(1 << 32) + 8192), dict(original=1 << 31), dict(rot=(1 << 32) + 64)):
        with pytest.raises(ValueError, match="32-bit"):
            santa.rope_table(**{"rot": 64, "scaling": "bands", "factor": 2.0, "device": "cpu", **bad})
    for rot in (65538, (1 << 31) - 2, -2, 0):
        with pytest.raises(santa.SantaError):
            santa.rope_table(rot, device="cpu")
    assert santa.rope_table(64, scaling="bands", factor=2.0, original=(1 << 31) - 1, device="cpu").rot == 64
