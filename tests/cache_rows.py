"""Attention in 64 bits with a bar for each row, small enough to miss a block of keys.

A row's output is o = sum_j p_j v_j. Its bar is on the norm of the error over the row's d values:
  - the weights are rounded before their product with v, each by at most half a step of bf16, 2^-8 of itself. Roundings of
    different keys go either way, so they add up as sqrt(sum_j p_j^2 |v_j|^2) 2^-8; taking the largest possible rounding for the
    usual one and four times the sum leaves more than six of its standard deviations, and holds for a single key too;
  - o is rounded once to bf16: each value by at most 2^-8 of itself, |o| 2^-8 together;
  - scores and exponentials in fp32: a score of magnitude below 2^5 is off by about 2^-24 sqrt(d) 2^5 / sqrt(d), 2^-19 of
    its weight, the hardware's exponential by 2^-22: 2^-18 sum_j p_j |v_j|.
test_cache_rows_cpu.py shows that losing any 16 keys, or counting them twice, is more than this.
"""
import torch

# B, H, Hkv, d, page, S (keys of the longest sequence), T, window, sinks
LONG = [
    (1, 4, 4, 64, 64, 2100, 1, 0, 0), (2, 8, 2, 128, 16, 4000, 1, 0, 0), (1, 16, 1, 64, 128, 9000, 1, 0, 0),
    (3, 8, 2, 128, 128, 9000, 2, 0, 0), (1, 4, 2, 128, 32, 8000, 7, 3000, 20),
    (1, 8, 2, 64, 64, 4000, 40, 0, 0), (2, 8, 2, 128, 16, 9000, 33, 0, 0), (1, 8, 2, 64, 64, 8000, 256, 0, 0),
    (1, 8, 2, 128, 32, 8000, 140, 2500, 30),
]


def inputs(B, H, Hkv, d, S, T, seed):
    """q [B, H, T, d], k and v [B, Hkv, S, d], bf16 on the CPU."""
    G = torch.Generator().manual_seed(seed)
    return [torch.randn(*s, generator=G).to(torch.bfloat16) for s in ((B, H, T, d), (B, Hkv, S, d), (B, Hkv, S, d))]


def starts_of(B, S, T):
    return [S - T - b * (S - T) // 3 for b in range(B)]


def weights(q, k, start, window=0, sinks=0, scale=None):
    """p [H, T, S] of one sequence: q [H, T, d], k [Hkv, S, d]."""
    H, T, d = q.shape
    z = q.double() @ k.double().repeat_interleave(H // k.shape[0], 0).mT * (d**-0.5 if scale is None else scale)
    p = start + torch.arange(T, device=q.device)[:, None]
    j = torch.arange(k.shape[1], device=q.device)
    seen = j <= p
    if window:
        seen = seen & ((j > p - window) | (j < sinks))
    z = z.masked_fill(~seen, -float("inf"))
    return torch.softmax(z, -1).nan_to_num(0.0)  # a row that sees nothing


def attend(q, k, v, starts, window=0, sinks=0, scale=None):
    """o [B, H, T, d] in 64 bits and the bars [B, H, T]."""
    out, bars = [], []
    for b, start in enumerate(starts):
        p = weights(q[b], k[b], int(start), window, sinks, scale)
        vv = v[b].double().repeat_interleave(q.shape[1] // v.shape[1], 0)
        o, n = p @ vv, vv.norm(dim=-1)[..., None]
        bars.append(4 * 2**-8 * ((p * p) @ (n * n))[..., 0].sqrt() + 2**-8 * o.norm(dim=-1) + 2**-18 * (p @ n)[..., 0] + 1e-30)
        out.append(o)
    return torch.stack(out), torch.stack(bars)


def worst(got, want, bars):
    """The largest row error in units of its bar."""
    off = (got.double() - want).norm(dim=-1) / bars
    return float(torch.where(off.isfinite(), off, torch.full_like(off, float("inf"))).max())
