"""The rows' bars of cache_rows see any 16 keys that are lost or counted twice."""
import pytest
import torch

import cache_ref
import cache_rows


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", [c for c in cache_rows.LONG if c[6] <= 40 and c[0] == 1], ids=str)
def test_a_lost_block_of_16_keys_shows(case, dtype):
    B, H, Hkv, d, page, S, T, window, sinks = case
    q, k, v = cache_rows.inputs(B, H, Hkv, d, S, T, S)
    if dtype == "e4m3":
        k, v = cache_ref.quantise(k), cache_ref.quantise(v)
    starts = cache_rows.starts_of(B, S, T)
    want, bars = cache_rows.attend(q, k, v, starts, window, sinks)
    p = cache_rows.weights(q[0], k[0], starts[0], window, sinks)
    heads = v[0].double().repeat_interleave(H // Hkv, 0)
    for j in range(0, S - 15, 16):
        block = p[..., j : j + 16]
        mass = block.sum(-1, keepdim=True)
        if not (mass > 0).all():  # before the window
            continue
        part = block @ heads[:, j : j + 16]
        for sign in (-1, 1):  # lost, counted twice
            got = (want[0] + sign * part) / (1 + sign * mass)
            # a block belongs to all rows of a key/value head
            off = ((got - want[0]).norm(dim=-1) / bars[0]).reshape(Hkv, -1).amax(-1)
            assert off.min() > 1, (j, sign, float(off.min()))


def test_the_rounding_alone_stays_far_below():
    """Weights and outputs rounded to bf16 in exact arithmetic."""
    B, H, Hkv, d, page, S, T, window, sinks = cache_rows.LONG[0]
    q, k, v = cache_rows.inputs(B, H, Hkv, d, S, T, 1)
    starts = cache_rows.starts_of(B, S, T)
    want, bars = cache_rows.attend(q, k, v, starts)
    p = cache_rows.weights(q[0], k[0], starts[0])
    e = p / p.amax(-1, keepdim=True)
    got = (e.to(torch.bfloat16).double() @ v[0].double()) / e.sum(-1, keepdim=True)
    assert cache_rows.worst(got[None].to(torch.bfloat16), want, bars) < 0.5
