"""Attention over long caches, whose keys several CTAs share, against cache_rows: each row within a bar that a lost or doubled
block of 16 keys breaks."""
import pytest
import torch

import cache_ref
import cache_rows
from titans_long_term_b200 import PagedCache

pytestmark = pytest.mark.gpu


def filled(B, H, d, dtype, page, k, v, seed):
    """A cache with k, v [B, Hkv, S, d] in scattered pages, and the values that it stands for."""
    S, G = k.shape[2], torch.Generator().manual_seed(seed)
    most = -(-S // page)
    cache = PagedCache(d, dtype, B, H, kv_heads=k.shape[1], page=page, num_pages=B * most + 2, max_pages=most)
    pages = cache.new_pages()
    table = torch.randperm(B * most + 2, generator=G)[: B * most].to(torch.int32).reshape(B, most).cuda()
    cache.append(k, v, pages, table, torch.zeros(B, dtype=torch.int32, device="cuda"))
    if dtype == "e4m3":
        k, v = cache_ref.quantise(k), cache_ref.quantise(v)
    return cache, pages, table, k, v


def check(cache, pages, table, q, k, v, starts, window=0, sinks=0):
    at = torch.tensor(starts, dtype=torch.int32, device="cuda")
    o = cache.attend(q, pages, table, at, window=window, sinks=sinks)
    cache.sync_status()
    want, bars = cache_rows.attend(q, k, v, starts, window, sinks)
    assert cache_rows.worst(o, want, bars) <= 1


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", cache_rows.LONG, ids=str)
def test_long_caches(case, dtype):
    B, H, Hkv, d, page, S, T, window, sinks = case
    q, k, v = (x.cuda() for x in cache_rows.inputs(B, H, Hkv, d, S, T, S))
    cache, pages, table, k, v = filled(B, H, d, dtype, page, k, v, S)
    check(cache, pages, table, q, k, v, cache_rows.starts_of(B, S, T), window, sinks)
