"""Value rows that carry weight but no value (no-op sinks, padding), and value rows of very unlike size: the others keep
their precision, relative to the output's own size (cache_rows)."""
import pytest
import torch

import cache_rows
from test_cache_rows_gpu import check, filled

pytestmark = pytest.mark.gpu


def with_null_keys(B, H, Hkv, d, S, T, where, weight, size, seed):
    """q, k, v whose keys at `where` have zero values and, over all rows of a head, about `weight` of the weights together;
    the other values are of magnitude `size`."""
    q, k, v = cache_rows.inputs(B, H, Hkv, d, S, T, seed)
    v = (v.float() * size).to(torch.bfloat16)
    q[..., 0] = 4.0  # a direction that only the null keys use
    k[..., 0] = 0.0
    rest = 1.6 * S / len(where)  # sum of exp(q.k / sqrt(d)) over the others, N(0, 1) scores
    height = torch.log(torch.tensor(weight / (1 - weight) * rest)) * d**0.5 / 4
    k[:, :, where] = 0.0
    v[:, :, where] = 0.0
    k[:, :, where, 0] = height.to(torch.bfloat16)
    return q.cuda(), k.cuda(), v.cuda()


@pytest.mark.parametrize("dtype", ["e4m3", "bf16"])
@pytest.mark.parametrize("weight", [0.26, 0.9, 0.986, 0.9999])
@pytest.mark.parametrize("B,H,Hkv,d,S,T,where,size", [
    (1, 4, 1, 128, 2001, 1, [0], 1.0), (2, 16, 2, 64, 8192, 1, [0], 0.01), (1, 8, 1, 128, 3000, 2, [1500], 1.0),
    (3, 8, 8, 64, 700, 5, [0, 1, 2, 3, 333, 690], 1e-4), (1, 8, 2, 128, 3000, 20, [0, 17], 0.01)])
def test_keys_without_a_value(B, H, Hkv, d, S, T, where, size, weight, dtype):
    q, k, v = with_null_keys(B, H, Hkv, d, S, T, where, weight, size, S)
    cache, pages, table, k, v = filled(B, H, d, dtype, 32, k, v, S)
    check(cache, pages, table, q, k, v, cache_rows.starts_of(B, S, T))


@pytest.mark.parametrize("T", [1, 4, 40])
def test_a_head_without_any_value(T):
    q, k, v = (x.cuda() for x in cache_rows.inputs(2, 4, 2, 64, 900, T, T))
    v[:, 0] = 0
    cache, pages, table, k, v = filled(2, 4, 64, "e4m3", 16, k, v, T)
    check(cache, pages, table, q, k, v, [900 - T, 500])


@pytest.mark.parametrize("dtype", ["e4m3", "bf16"])
@pytest.mark.parametrize("H,T", [(4, 1), (16, 1), (4, 30)])
@pytest.mark.parametrize("low,high", [(-4, 4), (-30, 0), (0, 30), (-30, 30)])
def test_values_of_unlike_size(low, high, H, T, dtype):
    """Powers of ten, key by key: the largest values' keys are the output, whatever their place in the cache."""
    S = 3000
    q, k, v = cache_rows.inputs(2, H, 1, 128, S, T, S + T)
    G = torch.Generator().manual_seed(H)
    v = (v.double() * 10 ** (low + (high - low) * torch.rand(2, 1, S, 1, generator=G).double())).to(torch.bfloat16)
    cache, pages, table, k, v = filled(2, H, 128, dtype, 64, k.cuda(), v.cuda(), 1)
    check(cache, pages, table, q.cuda(), k, v, [S - T, 1000])


@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("boost", [40.0, 200.0, 2000.0])
def test_a_null_key_far_above_the_others(T, boost):
    """Scores of the null key higher than any exponent of a float: what is left of the others is 0 or tiny, never NaN, and a row
    that sees it only with a neighbour of the same height keeps that one's half."""
    q, k, v = cache_rows.inputs(1, 4, 1, 128, 600, T, 3)
    q[..., 0], k[..., 0] = 8.0, 0.0
    k[:, :, 100, 0] = boost
    v[:, :, 100] = 0
    k[:, :, 101] = k[:, :, 100]
    cache, pages, table, k, v = filled(1, 4, 128, "e4m3", 16, k.cuda(), v.cuda(), 1)
    check(cache, pages, table, q.cuda(), k, v, [600 - T])
    k2 = k.clone()
    k2[:, :, 101] = 0  # alone
    cache, pages, table, k2, v = filled(1, 4, 128, "e4m3", 16, k2.to(torch.bfloat16), v.to(torch.bfloat16), 1)
    check(cache, pages, table, q.cuda(), k2, v, [600 - T])
