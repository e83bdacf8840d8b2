"""Sizes past 32 bits, which C arguments would take the low bits of, and tensors of another device: refused
by the calls over a paged cache before anything is enqueued."""
import pytest
import torch

from stochastic_sparse_kv_gb300 import santa

pytestmark = pytest.mark.gpu
DEV = "cuda"
bf16 = torch.bfloat16


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def small(columns=4, page=16, H_kv=2):
    cache = santa.new_paged_cache(4, H_kv, page, 64, 1, columns)
    cache.table[:, :4] = torch.arange(4)
    return cache


@pytest.mark.parametrize("T", [(1 << 30) + 3, (1 << 31) + 3, (1 << 32) + 3])
def test_tokens(T):
    """One row stands for them all (token stride 0), three of them live."""
    cache, row = small(), torch.ones(1, 1, 2, 64, dtype=bf16, device=DEV)
    many = row.expand(1, T, 2, 64)
    for call in (lambda: santa.paged_append(cache, many, many, ints([0]), ints([3])),
                 lambda: santa.attend_paged(many, cache, ints([0]), ints([3])),
                 lambda: santa.rope(many, santa.rope_table(64), ints([0]), ints([3]), out=many)):
        with pytest.raises(santa.SantaError) as e:
            call()
        assert e.value.status == santa.ERR_UNSUPPORTED
    assert not cache.k.any() and not cache.v.any()


def test_heads():
    cache, row = small(), torch.ones(1, 1, 1, 64, dtype=bf16, device=DEV)
    many = row.expand(1, 1, (1 << 32) + 2, 64)
    new = torch.ones(1, 1, 2, 64, dtype=bf16, device=DEV)
    for call in (lambda: santa.attend_paged(many, cache, ints([0])),
                 lambda: santa.rope(many, santa.rope_table(64), ints([0]), out=many),
                 lambda: santa.paged_append(cache, new, new, ints([0]), rope=santa.rope_table(64), q=many, q_out=many)):
        with pytest.raises(santa.SantaError):
            call()
    assert not cache.k.any() and not cache.v.any()


def test_columns():
    """A table of 2^24 + 1 columns of pages of 256: 2^32 + 256 positions, of which C would see 256."""
    cache, new = small((1 << 24) + 1, 256), torch.ones(1, 1, 2, 64, dtype=bf16, device=DEV)
    for call in (lambda: santa.attend_paged(new, cache, ints([0])), lambda: santa.paged_append(cache, new, new, ints([0]))):
        with pytest.raises(santa.SantaError) as e:
            call()
        assert e.value.status == santa.ERR_UNSUPPORTED
    assert not cache.k.any() and not cache.v.any()


def test_a_workspace_of_another_device():
    """(the kernels would write to its address)"""
    cache, new, table = small(), torch.ones(1, 1, 2, 64, dtype=bf16, device=DEV), santa.rope_table(64)
    for ws in (torch.zeros(64 << 20, dtype=torch.uint8), torch.empty(64 << 20, dtype=torch.uint8, device="meta")):
        for call in (lambda: santa.rope(new, table, ints([0]), workspace=ws), lambda: santa.attend_paged(new, cache, ints([0]), workspace=ws),
                     lambda: santa.paged_append(cache, new, new, ints([0]), workspace=ws)):
            with pytest.raises(ValueError, match="workspace"):
                call()
    assert not cache.k.any() and not cache.v.any()
    # an empty one is too small, not none
    with pytest.raises(santa.SantaError):
        santa.attend_paged(new, cache, ints([0]), workspace=torch.empty(0, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("T", [1, 20, 150])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [150, 5000])
def test_a_result_at_16_bytes(T, d, n):
    """(rows of a result at a multiple of 32 bytes are stored 32 bytes at a time)"""
    g = torch.Generator(device=DEV).manual_seed(T)
    cols = -(-n // 16)
    k, v = (torch.randn(2 * cols, 2, 16, d, generator=g, device=DEV).to(bf16) for _ in range(2))
    cache = santa.PagedCache(k, v, torch.arange(2 * cols, device=DEV, dtype=torch.int32).view(2, cols))
    q = torch.randn(2, T, 8, d, generator=g, device=DEV).to(bf16)
    pos, counts = ints([n - T, 0]), ints([T, T - T // 3])
    want = santa.attend_paged(q, cache, pos, counts)
    room = torch.full((q.numel() + 16,), 7.0, dtype=bf16, device=DEV)
    out = room[8:-8].view_as(q)
    assert out.data_ptr() % 32 == 16
    santa.attend_paged(q, cache, pos, counts, out=out)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1, :T - T // 3], want[1, :T - T // 3])
    assert (out[1, T - T // 3:] == 7).all() and (room[:8] == 7).all() and (room[-8:] == 7).all()
    with pytest.raises(santa.SantaError):
        santa.attend_paged(q, cache, pos, counts, out=room[4:-12].view_as(q))
