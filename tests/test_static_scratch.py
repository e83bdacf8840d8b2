"""The size limit of santa_decode_static: 16 MiB behind the control block."""
import ctypes

import pytest
import torch

from stochastic_sparse_kv_gb300 import santa, _build, workloads


def largest_keys():
    """The longest cache (multiples of 32) of one row and 32 heads whose weights and chunk data fill
    16 MiB, beside the 512 bytes of counters that such a problem needs."""
    sh = lambda n: santa.make_shape(1, 32, 8, 128, n)  # noqa: E731
    per = santa.workspace_size(sh(96000), 256, "systematic") - santa.workspace_size(sh(64000), 256, "systematic")
    base = santa.workspace_size(sh(64000), 256, "systematic") - 65536 + 512
    return 64000 + ((16 << 20) - base) * 32000 // per // 32 * 32


def test_a_problem_of_16_mib_is_accepted():
    _build.build()
    lib = santa.load()
    n = largest_keys()
    assert 100000 < n < 130000
    vp = ctypes.c_void_p

    def call(keys):  # without a query: refused as such when the size is not
        return lib.santa_decode_static(ctypes.byref(santa.make_shape(1, 32, 8, 128, keys)), vp(0), vp(4096), vp(4096),
                                       vp(4096), 256, santa.SYSTEMATIC, ctypes.c_uint64(0), vp(4096), vp(0), vp(0))

    assert call(n) == -1
    assert call(n + 2048) == santa.ERR_SCRATCH
    size = santa.workspace_size(santa.make_shape(1, 32, 8, 128, n), 256, "systematic")
    assert (16 << 20) < size <= santa.STATIC_SCRATCH_BYTES


@pytest.mark.gpu
def test_a_problem_of_16_mib_runs():
    lib = santa.load()
    n = largest_keys()
    _, q, k, v, sl = workloads.small("static", 1, 32, 8, 128, n, 256, seq_lens=[n], seed=9)
    q, k, v, sl = (x.cuda() for x in (q, k, v, sl))
    out = torch.empty(1, 32, 128, device="cuda")
    idx = torch.empty(1, 32, 256, dtype=torch.int32, device="cuda")
    p = [ctypes.c_void_p(x.data_ptr()) for x in (q, k, v, sl, out, idx)]
    rc = lib.santa_decode_static(ctypes.byref(santa.make_shape(1, 32, 8, 128, n)), *p[:4], 256, santa.SYSTEMATIC,
                                 ctypes.c_uint64(3), p[4], p[5], ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0
    want, widx = santa.decode(q, k, v, sl, 256, "systematic", seed=3)
    torch.cuda.synchronize()
    assert torch.equal(idx, widx) and torch.equal(out, want)
