"""The bounded waits of attention over a paged cache, as in test_zz_timeout.py: with a 1 ns limit
the warps give up, the call reports SANTA_DEV_TIMEOUT, copies in flight are waited for, the arrival
counters of pieces are zero again, and the next call gives the same result as before."""
import pytest
import torch

from stochastic_sparse_kv_gb300 import santa

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("B,T,n", [(1, 1, 30000), (3, 200, 2000), (2, 20, 5000)])
@pytest.mark.parametrize("d", [64, 128])
def test_short_wait_limit_reports_a_timeout_and_leaves_the_context_usable(B, T, n, d):
    g = torch.Generator(device=DEV).manual_seed(T)
    page, H_kv, G = 64, 4, 4
    cols = -(-n // page)
    k, v = (torch.randn(B * cols, H_kv, page, d, generator=g, device=DEV).bfloat16() for _ in range(2))
    table = torch.randperm(B * cols, generator=g, device=DEV).view(B, cols).to(torch.int32)
    q = torch.randn(B, T, H_kv * G, d, generator=g, device=DEV).bfloat16()
    pos = torch.full((B,), n - T, dtype=torch.int32, device=DEV)
    ws = santa.new_workspace(64 << 20, DEV)
    call = lambda: santa.attend_paged(q, santa.PagedCache(k, v, table), pos, workspace=ws)  # noqa: E731
    ref = call()
    torch.cuda.synchronize()
    assert santa.device_status(ws) == 0
    try:
        santa.set_wait_limit(1)  # 1 ns: the first wait that is not already satisfied gives up
        for _ in range(3):
            call()
        torch.cuda.synchronize()
        code = santa.device_status(ws)
    finally:
        santa.set_wait_limit(0)
    assert code == santa.DEV_TIMEOUT
    assert santa.device_status(ws) == 0  # cleared by the read
    assert not ws[256:65536].any()       # every arrival counter
    for _ in range(3):
        assert torch.equal(call(), ref)
    assert santa.device_status(ws) == 0
