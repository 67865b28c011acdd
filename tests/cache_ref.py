"""The paged cache and its attention in 64 bits, key by key from the definition."""
import torch


def quantise(x):
    """x [.., d] -> the values an e4m3 cache stands for: 4 significant bits at the smallest power-of-two scale."""
    x = x.double()
    top = torch.where(x.isfinite(), x.abs(), torch.zeros_like(x)).amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(top > 0, top, torch.full_like(top, 448.0)) / 448)).clamp(min=-117)
    y = (x / torch.exp2(e)).clamp(-448, 448)
    ulp = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0**-6))) - 3)
    return torch.round(y / ulp) * ulp * torch.exp2(e)


def attend(q, k, v, starts, counts, window=0, sinks=0, scale=None, missing=None):
    """q [B, H, T, d]; k, v [B, Hkv, S, d] by position; missing [B, S]: keys that no row sees."""
    B, H, T, d = q.shape
    scale = d**-0.5 if scale is None else scale
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    j = torch.arange(k.shape[2], device=q.device)
    for b in range(B):
        for t in range(int(counts[b])):
            p = int(starts[b]) + t
            seen = j <= p
            if window:
                seen &= (j > p - window) | (j < sinks)
            if missing is not None:
                seen &= ~missing[b]
            if not seen.any():
                continue
            rep = H // k.shape[1]
            kk, vv = (x[b, :, seen].double().repeat_interleave(rep, 0) for x in (k, v))
            z = (kk @ q[b, :, t].double()[..., None])[..., 0] * scale
            p_ = torch.softmax(z, -1)
            out[b, :, t] = (p_[:, None] @ vv)[:, 0]
    return out


def bar(want, v):
    """A bf16 output: half a step of itself, and the weights' rounding to bf16 before their product with v, 2^-8 of
    each term at most: the terms' absolute values sum to at most max |v|, and a weight's rounding averages out over
    the terms, but one key may carry all of it, so the whole of it stands here."""
    return 2**-8 * want.abs() + 2**-8 * v.double().abs().amax() + 1e-30
