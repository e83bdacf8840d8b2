"""Attention over a paged cache with wait limits around the time that its waits take (1 to 8 us run out in
most of the shapes): some run out with copies and products under way and pieces written by some CTAs and not by
others; at 1 ns all do, at 2 ms none.  Whatever ran out, the
call ends, reports it, leaves the arrival counters at zero, and the next call gives the same bits as
before.  The waits give up by themselves: nothing faults."""
import pytest
import torch

from stochastic_sparse_kv_gb300 import santa

pytestmark = pytest.mark.gpu
DEV = "cuda"
LIMITS_NS = [1, 1000, 1300, 1700, 2200, 3000, 4000, 5500, 7500, 10000, 14000, 20000, 50000, 200000, 2000000]


@pytest.mark.parametrize("B,T,n,window", [(1, 1, 30000, 0), (16, 1, 9000, 0), (3, 200, 2000, 0), (2, 20, 5000, 0), (1, 700, 6000, 0),
                                          (6, 130, 1500, 300), (40, 1, 40000, 0), (12, 100, 80000, 0)])
@pytest.mark.parametrize("d", [64, 128])
def test_limits_around_what_the_waits_take(B, T, n, window, d):
    g = torch.Generator(device=DEV).manual_seed(T + d)
    page, H_kv, G = 64, 4, 4
    cols = -(-n // page)
    k, v = (torch.randn(min(B * cols, 4000), H_kv, page, d, generator=g, device=DEV).bfloat16() for _ in range(2))
    table = (torch.randperm(B * cols, generator=g, device=DEV) % 4000).view(B, cols).to(torch.int32)
    q = torch.randn(B, T, H_kv * G, d, generator=g, device=DEV).bfloat16()
    pos = torch.full((B,), n - T, dtype=torch.int32, device=DEV)
    ws = santa.new_workspace(64 << 20, DEV)
    flush = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)
    cache = santa.PagedCache(k, v, table)
    call = lambda: santa.attend_paged(q, cache, pos, window=window, sinks=3, workspace=ws)  # noqa: E731
    ref = call()
    torch.cuda.synchronize()
    assert santa.device_status(ws) == 0
    codes = []
    try:
        for limit in LIMITS_NS:
            for cold in (True, False):
                if cold:
                    flush.fill_(limit & 0x7f)
                santa.set_wait_limit(limit)
                out = call()
                torch.cuda.synchronize()
                codes.append(santa.device_status(ws))
                assert codes[-1] in (0, santa.DEV_TIMEOUT)
                assert not ws[256:65536].any(), f"arrival counters after a limit of {limit} ns"
                assert codes[-1] or torch.equal(out, ref)
                santa.set_wait_limit(0)
                assert torch.equal(call(), ref)
                assert santa.device_status(ws) == 0
    finally:
        santa.set_wait_limit(0)
    print("timeouts:", [limit for limit, a, b in zip(LIMITS_NS, codes[::2], codes[1::2]) if a or b])
    assert codes[:2] == [santa.DEV_TIMEOUT] * 2 and codes[-2:] == [0, 0]
