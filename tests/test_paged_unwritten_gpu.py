"""Rows of a result that no live token writes, where the result is the call's own: zeros, whatever the
memory held, also without counts and for batch rows that are skipped.  And the flag for it in the C ABI,
with a result given."""
import ctypes

import pytest
import torch

from stochastic_sparse_kv_gb300 import santa

pytestmark = pytest.mark.gpu
DEV = "cuda"
bf16 = torch.bfloat16
BIG = (1 << 31) - 1


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.fixture(autouse=True)
def soiled(monkeypatch):
    """The memory that a call allocates for its result holds sevens."""
    monkeypatch.setattr(santa, "_out_rows", lambda x, *_: torch.full(x.shape, 7.0, dtype=bf16, device=x.device))


def problem(B, T, H_kv, G, d, page, columns, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    k, v = (torch.randn(B * columns, H_kv, page, d, generator=g, device=DEV).to(bf16) for _ in range(2))
    table = torch.arange(B * columns, device=DEV, dtype=torch.int32).view(B, columns)
    q, k_new, v_new = (torch.randn(B, T, h, d, generator=g, device=DEV).to(bf16) for h in (H_kv * G, H_kv, H_kv))
    return q, k_new, v_new, santa.PagedCache(k, v, table)


def expect(got, given, live):
    """`got`: zeros but for the first live[b] tokens of each batch row, which are those of `given`, a result
    over rows of sevens."""
    for b, n in enumerate(live):
        assert torch.equal(got[b, :n], given[b, :n])
        assert not got[b, n:].any(), f"batch row {b}"
        assert (given[b, n:] == 7).all()
        assert n == 0 or got[b, :n].any()


CASES = [(1, 64, 1), (1, 128, 4), (3, 128, 8), (40, 64, 4), (150, 128, 2), (600, 64, 1)]   # T, d, G


@pytest.mark.parametrize("T,d,G", CASES)
@pytest.mark.parametrize("counted", [False, True])
def test_attend(T, d, G, counted):
    B, page, columns = 5, 64, 12
    q, _, _, cache = problem(B, T, 2, G, d, page, columns)
    n_max = page * columns
    pos = ints([3, -1, n_max - T + 1, n_max - T, BIG])
    live = [T, 0, 0, T, 0]
    counts = None
    if counted:
        counts, live = ints([T // 2, T, T, 0, T]), [T // 2, 0, 0, 0, 0]
    given = torch.full_like(q, 7.0)
    santa.attend_paged(q, cache, pos, counts, out=given)
    ws = santa.new_workspace(64 << 20, DEV)
    for workspace in (None, ws):
        got = santa.attend_paged(q, cache, pos, counts, workspace=workspace)
        expect(got, given, live)
    assert santa.device_status(ws) == santa.DEV_BAD_POSITION


@pytest.mark.parametrize("T,d,G", CASES)
@pytest.mark.parametrize("layout,rot", [("halves", 16), ("pairs", 64)])
@pytest.mark.parametrize("counted", [False, True])
def test_rope_and_append(T, d, G, layout, rot, counted):
    B, page, columns = 5, 64, 12
    q, k_new, v_new, cache = problem(B, T, 2, G, d, page, columns)
    table = santa.rope_table(rot, layout=layout)
    n_max = page * columns
    counts = ints([T // 2, T, T, 0, T]) if counted else None
    # alone: positions up to the largest there is
    pos = ints([3, -1, BIG - T + 1, BIG - T, BIG])
    live = [T // 2, 0, 0, 0, 0] if counted else [T, 0, 0, T, 0]
    given = torch.full_like(q, 7.0)
    santa.rope(q, table, pos, counts, out=given)
    got = santa.rope(q, table, pos, counts)
    expect(got, given, live)
    # with K and V: positions of the cache; what is held is the same with q's rows given and with the call's own
    pos = ints([3, -1, n_max - T + 1, n_max - T, BIG])
    held = [x.clone() for x in cache[:2]]
    given.fill_(7.0)
    santa.paged_append(cache, k_new, v_new, pos, counts, rope=table, q=q, q_out=given)
    other = santa.PagedCache(*held, cache.table)
    got = santa.paged_append(other, k_new, v_new, pos, counts, rope=table, q=q)
    expect(got, given, live)
    assert torch.equal(other.k, cache.k) and torch.equal(other.v, cache.v)


def test_a_call_with_no_live_token_at_all():
    """Every row skipped or of count 0, one to thousands of dead tokens."""
    for B, T in ((1, 1), (7, 3), (2, 3000)):
        q, _, _, cache = problem(B, T, 2, 4, 128, 64, 2)
        table = santa.rope_table(128)
        for pos, counts in (([-1] * B, None), ([0] * B, [0] * B), ([5] * B, [T + 1] * B)):
            counts = ints(counts) if counts else None
            for call in (lambda: santa.attend_paged(q, cache, ints(pos), counts), lambda: santa.rope(q, table, ints(pos), counts)):
                assert not call().any()


def test_the_flag_over_a_strided_result_given():
    """In the C ABI: rows of a padded result become zeros, the padding between them stays."""
    B, T, H, d = 3, 21, 5, 64
    x = torch.randn(B, T, H, d, device=DEV).to(bf16)
    room = torch.full((B, T, H, d + 8), 7.0, dtype=bf16, device=DEV)
    out = room[..., :d]
    i64 = ctypes.c_int64 * 3
    table = santa.rope_table(32)
    rotation = santa._Rotation(table.turns.data_ptr(), 32, 0, 1.0)
    pos, counts = ints([4, 9, -5]), ints([8, 21, 3])
    want = santa.rope(x, table, pos, counts)
    torch.cuda.synchronize()
    rc = santa.load().santa_rope(B, T | santa.CLEAR_REST, H, d, x.data_ptr(), i64(*x.stride()[:3]), out.data_ptr(),
                                 i64(*out.stride()[:3]), ctypes.byref(rotation), pos.data_ptr(), counts.data_ptr(), None,
                                 torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    assert torch.equal(out, want) and not out[0, 8:].any() and not out[2].any() and out[1].any()
    assert (room[..., d:] == 7).all()


def test_captured():
    """The rest becomes zeros at every replay, by the counts of that replay."""
    B, T = 3, 70
    q, _, _, cache = problem(B, T, 2, 4, 64, 16, 40)
    pos, counts = ints([100, 200, 300]), ints([T, T, T])
    santa.attend_paged(q, cache, pos, counts)   # warm
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = santa.attend_paged(q, cache, pos, counts)
    for live in ([T, T, T], [5, 0, T], [T, 1, 2]):
        counts.copy_(ints(live))
        graph.replay()
        given = torch.full_like(q, 7.0)
        santa.attend_paged(q, cache, pos, counts, out=given)
        expect(out, given, live)


@pytest.mark.parametrize("T,H_kv,d", [(2, 1, 64), (9, 2, 128), (200, 1, 64)])
def test_many_batch_rows_few_of_them_padded(T, H_kv, d):
    """Groups of 32 batch rows with none, one and all padded or skipped."""
    B = 150
    q, _, _, cache = problem(B, T, H_kv, 4, d, 16, 20)
    live = [T] * B
    pos = [(7 * b) % 100 for b in range(B)]
    for b in (40, *range(64, 96), 149):
        live[b] = b % T
    pos[100] = -1
    counts = ints(live)
    live[100] = 0
    given = torch.full_like(q, 7.0)
    santa.attend_paged(q, cache, ints(pos), counts, out=given)
    expect(santa.attend_paged(q, cache, ints(pos), counts), given, live)
