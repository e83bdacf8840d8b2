"""Prompts in chunks and single tokens through append and attention, element by element: the rotated rows against
their formula, and each result against 64 bits over what the cache and the queries then hold."""
import pytest
import torch

from stochastic_sparse_kv_gb300 import santa
from tests import paged_util as pu
from tests.test_paged_gpu import check, check_rope, f64, gen, ints, rand

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("d,G,page,layout,window,sinks", [(128, 4, 64, "halves", 0, 0), (64, 2, 16, "pairs", 0, 0), (64, 8, 32, "halves", 60, 3),
                                                          (128, 1, 128, "pairs", 33, 0)])
@pytest.mark.parametrize("chunk", [48, 150])
def test_chunks_then_single_tokens(d, G, page, layout, window, sinks, chunk):
    g = gen(d + G + chunk)
    B, H_kv, lens = 4, 2, [310, 101, 49, 0]
    H_q, total = H_kv * G, max(lens)
    t = santa.rope_table(d, 500000.0, layout, "bands", 8.0, original=64)
    f, _ = pu.frequencies(d, 500000.0, "bands", 8.0, original=64)
    cols = -(-(total + 4) // page)
    table, n_pages = pu.pages(g, [n + 4 for n in lens], page, cols)
    cache = santa.new_paged_cache(n_pages, H_kv, page, d, B, cols)
    cache.table.copy_(table)
    pos = [0] * B
    steps = [[max(0, min(chunk, n - at)) for n in lens] for at in range(0, total, chunk)] + [[1] * B] * 3
    for counts in steps:
        T = chunk if max(counts) > 1 else 1
        q, k, v = (rand(g, B, T, h, d).to(DEV) for h in (H_q, H_kv, H_kv))
        turned = santa.paged_append(cache, k, v, ints(pos), ints(counts), rope=t, q=q)
        check_rope(turned, q.cpu(), f, 1.0, layout, pos, counts, torch.zeros_like(turned))
        held = torch.stack([torch.stack([cache.k[int(table[b, (pos[b] + i) // page]), :, (pos[b] + i) % page] if i < counts[b] else
                                         torch.zeros_like(k[b, i]) for i in range(T)]) for b in range(B)])
        check_rope(held, k.cpu(), f, 1.0, layout, pos, counts, torch.zeros_like(held))
        out = santa.attend_paged(turned, cache, ints(pos), ints(counts), window, sinks)
        want, spread = pu.attention(turned, cache.k.cpu(), cache.v.cpu(), table, pos, counts, window, sinks)
        check(out, want, spread, counts, torch.zeros_like(out))
        pos = [p + c for p, c in zip(pos, counts)]
    for b in range(B):
        assert pos[b] == lens[b] + 3
    assert f64(cache.v).any()
