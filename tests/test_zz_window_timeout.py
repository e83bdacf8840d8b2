"""The bounded waits of the bf16 windowed attention kernel, as in test_zz_timeout.py: with a 1 ns
limit the warps give up, the call reports SANTA_DEV_TIMEOUT, copies in flight are waited for,
and the next call gives the reference result.  (The 4-bit kernel waits on no barrier of its
copies: its call is unaffected by the limit.)"""
import pytest
import torch

from stochastic_sparse_kv_gb300 import santa, workloads

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("op", ["kv4", "window"])
@pytest.mark.parametrize("B,window", [(1, 0), (4, 5000)])
def test_short_wait_limit_reports_a_timeout_and_leaves_the_context_usable(op, B, window):
    seq = [16384, 16384, 9000, 16384][:B]
    _, q, k, v, sl = workloads.small("timeout", B, 32, 8, 128, 16384, 256, seq_lens=seq, seed=31)
    qd, kd, vd, sld = q.to(DEV), k.to(DEV), v.to(DEV), sl.to(DEV)
    ws = santa.new_workspace(32 << 20, DEV)
    if op == "kv4":
        cache = santa.new_kv4_cache(B, 8, 16384, 128)
        santa.kv4_append(cache, kd.transpose(1, 2), vd.transpose(1, 2), torch.zeros(B, dtype=torch.int32, device=DEV))
        call = lambda: santa.decode_kv4(qd, cache, sld, window, 4, workspace=ws)  # noqa: E731
    else:
        call = lambda: santa.decode_window(qd, kd, vd, sld, window, 4, workspace=ws)  # noqa: E731
    ref = call()
    torch.cuda.synchronize()
    assert santa.device_status(ws) == 0
    try:
        santa.set_wait_limit(1)  # 1 ns: the first wait that is not already satisfied gives up
        call()
        torch.cuda.synchronize()
        code = santa.device_status(ws)
    finally:
        santa.set_wait_limit(0)
    assert code == (santa.DEV_TIMEOUT if op == "window" else 0)
    assert santa.device_status(ws) == 0  # cleared by the read
    assert torch.equal(call(), ref)
