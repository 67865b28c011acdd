"""An e4m3 cache of values near the largest bf16: what it holds is finite."""
import pytest
import torch

import cache_ref
from titans_long_term_b200 import PagedCache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
def test_the_largest_values_stay_finite(d):
    top = torch.finfo(torch.bfloat16).max
    x = torch.zeros(1, 1, 16, d)
    for t, f in enumerate((1.0, -1.0, 0.98, 0.97, 0.96, 0.95, 0.94, 0.9, 0.875, 0.87, 0.8, 0.75, 0.6, 0.51, 0.49, 0.25)):
        x[0, 0, t, 0], x[0, 0, t, 1], x[0, 0, t, 2] = f * top, f * top / 3, -f * top / 1000
    x[0, 0, 0, 3], x[0, 0, 2, 4] = float("inf"), -float("inf")
    x = x.to(torch.bfloat16).cuda()
    cache = PagedCache(d, "e4m3", 1, 1, page=16, num_pages=1, max_pages=1)
    pages, table, start = cache.new_pages(), *(torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((1, 1), (1,)))
    cache.append(x, x, pages, table, start)
    k, v = cache.read(pages, table, start, 16)
    assert torch.equal(k, v) and torch.isfinite(k).all()
    want = cache_ref.quantise(x).clamp(-240 * 2.0**120, 240 * 2.0**120)  # 2^128 would not be a bf16 any more
    assert torch.equal(k.double(), want)
    o = cache.attend(torch.zeros(1, 1, 1, d, dtype=torch.bfloat16, device="cuda"), pages, table, start)
    assert torch.equal(o[0, 0, 0], v[0, 0, 0])  # one key: its value
    cache.sync_status()
