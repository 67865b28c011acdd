"""The gated delta rule token by token in 64 bits, and the inputs and bars of its tests.

Bars. u = 2^-24. A state or gate gradient is a chain of about six products of length <= 128 in fp32 or in fp16
pieces of 22 bits: each is off by about (sqrt(128) u + 2^-22) of its norm, together sqrt(6) times that, 2.2e-6;
NORM32 = 1e-5 leaves a factor of four for the sums over the tokens. A bf16 output is that value rounded once, half a
step 2^-8 of itself, after products whose operands hold 11 bits or more: four roundings of at most 2^-11 of the
largest value, 2^-9 of it.
"""
import torch

NORM32 = 1e-5


def inputs(B, H, Hk, T, d, mode, seed=0, device="cpu", ragged=False, reset=False, scale=1.0):
    """k, q of norm `scale`, v, g, beta, W; `ragged`: lengths from T down, one of them 0 and one 1 where B allows;
    `reset`: g = -inf at a few tokens."""
    G = torch.Generator().manual_seed(seed)
    tok = torch.bfloat16 if mode == "bf16" else torch.float32
    r = lambda *s: torch.randn(*s, generator=G)  # noqa: E731
    x = {n: (torch.nn.functional.normalize(r(B, Hk, T, d), dim=-1) * scale).to(tok) for n in ("k", "q")}
    x["v"] = r(B, H, T, d).to(tok)
    x["g"] = torch.log1p(-0.1 * torch.rand(B, H, T, generator=G))
    x["beta"] = torch.rand(B, H, T, generator=G)
    x["W"] = r(B, H, d, d) * 0.3
    x["dy"] = r(B, H, T, d).to(tok)
    x["dW"] = r(B, H, d, d) * 0.3
    x["attn"] = r(B, H, T, d).to(tok)
    if reset:
        x["g"][:, :, :: max(1, T // 3)] = -float("inf")
        x["beta"][:, :, :: max(1, T // 4)] = 0
    lengths = [T, 0, 1, T - 1, T // 2][:B] if ragged else [T] * B
    x["lengths"] = torch.tensor([max(0, n) for n in lengths], dtype=torch.int32)
    return {n: t.to(device) for n, t in x.items()}


def _heads(x):
    rep = x["v"].shape[1] // x["k"].shape[1]
    return {n: (x[n].repeat_interleave(rep, 1) if n in "kq" else x[n]).double() for n in ("k", "q", "v", "g", "beta")}


def forward(x, gated=False, keep=False):
    """y, W_T and, with keep, the states before every token."""
    t64, W, ys, states = _heads(x), x["W"].double(), [], []
    for t in range(x["v"].shape[2]):
        k, q, v, a, b = (t64[n][:, :, t] for n in ("k", "q", "v", "g", "beta"))
        live = (t < x["lengths"])[:, None, None]
        states.append(W)
        A = a.exp()[..., None, None] * W
        e = b[..., None] * (v - (A @ k[..., None])[..., 0])
        W = torch.where(live[..., None], A + e[..., None] * k[..., None, :], W)
        y = (W @ q[..., None])[..., 0]
        if gated:
            y = x["attn"][:, :, t].double() * torch.sigmoid(y)
        ys.append(torch.where(live, y, torch.zeros_like(y)))
    return (torch.stack(ys, 2), W, states) if keep else (torch.stack(ys, 2), W)


def backward(x):
    """Gradients of <dy, y> + <dW, W_T> by the adjoint of each token."""
    t64 = _heads(x)
    _, _, states = forward(x, keep=True)
    out = {n: torch.zeros_like(t) for n, t in t64.items()}
    dW = x["dW"].double()
    for t in reversed(range(x["v"].shape[2])):
        k, q, v, a, b = (t64[n][:, :, t] for n in ("k", "q", "v", "g", "beta"))
        dy = x["dy"][:, :, t].double()
        live = (t < x["lengths"])[:, None, None]
        A = a.exp()[..., None, None] * states[t]
        res = v - (A @ k[..., None])[..., 0]
        e = b[..., None] * res
        W = A + e[..., None] * k[..., None, :]
        F = dW + dy[..., None] * q[..., None, :]
        de = (F @ k[..., None])[..., 0]
        dA = F - (b[..., None] * de)[..., None] * k[..., None, :]
        one = {"q": (W.mT @ dy[..., None])[..., 0], "v": b[..., None] * de,
               "k": (F.mT @ e[..., None])[..., 0] - (A.mT @ (b[..., None] * de)[..., None])[..., 0],
               "beta": (de * res).sum(-1), "g": (dA * A).sum((-1, -2))}
        for n, z in one.items():
            keep = live if z.dim() == 3 else live[..., 0]
            out[n][:, :, t] = torch.where(keep, z, torch.zeros_like(z))
        dW = torch.where(live[..., None], a.exp()[..., None, None] * dA, dW)
    B, H, T, d = x["v"].shape
    for n in ("k", "q"):
        out[n] = out[n].reshape(B, x["k"].shape[1], -1, T, d).sum(2)
    return out | {"W": dW}


def assert_close(name, got, want, mode):
    """fp32 values by their norm per unit, bf16 values one by one (see the module's text)."""
    got, want = got.detach().double().cpu(), want.double().cpu()
    assert got.shape == want.shape and torch.isfinite(got).all(), name
    off = (got - want).flatten(2)
    ref = want.flatten(2)
    if mode == "fp32":
        bar = NORM32 * ref.norm(dim=-1) + 1e-30
        worst = (off.norm(dim=-1) / bar).max()
    else:
        bar = 2**-8 * ref.abs() + 2**-9 * ref.abs().amax(-1, keepdim=True) + 1e-30
        worst = (off.abs() / bar).max()
    assert worst <= 1, f"{name}: {float(worst):.3g} of the bar"
