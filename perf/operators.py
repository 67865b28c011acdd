"""The gated delta rule and the paged key/value cache with its attention: measured cases, the operators in
elementary torch arithmetic, and their definitions in 64 bits.

Gated delta rule, per (batch, head) unit with state W [d, d] (column convention M(x) = W x):
    A_t = exp(g_t) W_{t-1};  e_t = beta_t (v_t - A_t k_t);  W_t = A_t + e_t k_t^T;  y_t = W_t q_t.
H value heads share Hk key/query heads (head h reads key head h // (H / Hk)).

Paged cache, per (sequence, key/value head): token p of sequence b lies in page table[b, p // page], slot p % page. An
e4m3 cache keeps one power-of-two scale per token and head: the smallest 2^e with max |x| <= 448 * 2^e. Query t
of a chunk stands at p = starts[b] + t and sees keys j <= p with j > p - window (window 0: all) or j < sinks.
"""
import torch

own = False

CHUNK = 64


def listed():
    return [
        # A training batch's stream of 128 units, d = 64 (the 760M-class batch of this library's benchmark).
        dict(name="forward stream", op="forward", B=8, H=16, Hk=16, T=4096, d=64, dtype="bf16", ragged=False, gated=False),
        # Prefill of long prompts by the wide memory: 32 units, d = 128.
        dict(name="forward wide", op="forward", B=4, H=8, Hk=8, T=16384, d=128, dtype="bf16", ragged=False, gated=False),
        # A padded batch of short prompts, shared key heads, gating an attention branch.
        dict(name="forward ragged", op="forward", B=3, H=6, Hk=2, T=451, d=128, dtype="bf16", ragged=True, gated=True),
        # The fp32 mode on a short stream.
        dict(name="forward fp32", op="forward", B=2, H=4, Hk=4, T=1000, d=64, dtype="fp32", ragged=False, gated=False),
        # One token of one conversation: latency.
        dict(name="step one", op="step", B=1, H=16, Hk=16, T=1, d=64, dtype="bf16", ragged=False, gated=False),
        # One token of 64 conversations: the state's bandwidth.
        dict(name="step many", op="step", B=64, H=16, Hk=8, T=1, d=128, dtype="bf16", ragged=False, gated=True),
        # The training batch's backward pass.
        dict(name="backward stream", op="backward", B=8, H=16, Hk=16, T=4096, d=64, dtype="bf16", ragged=False, gated=False),
        # A padded batch's backward pass in fp32 with shared key heads.
        dict(name="backward ragged", op="backward", B=2, H=6, Hk=3, T=777, d=128, dtype="fp32", ragged=True, gated=False),
        # A prompt chunk written into an 8-bit cache and read back.
        dict(name="cache chunk", op="cache", B=8, H=4, Hk=4, T=1024, d=128, dtype="e4m3", S=6000, page=64, ragged=True),
        # One decoded token of 32 sequences written and read back.
        dict(name="cache token", op="cache", B=32, H=8, Hk=8, T=1, d=64, dtype="bf16", S=2048, page=16, ragged=False),
        # A chunk of new tokens over a long bf16 cache.
        dict(name="attend chunk", op="attend", B=2, H=16, Hk=4, T=2048, d=128, dtype="bf16", S=10000, page=64, window=0, sinks=0, ragged=False),
        # One token of 32 sequences over an 8-bit cache.
        dict(name="attend token", op="attend", B=32, H=16, Hk=4, T=1, d=128, dtype="e4m3", S=8192, page=64, window=0, sinks=0, ragged=False),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["forward", "forward", "step", "backward", "backward", "cache", "attend", "attend"])
    d = rng.choice([64, 128])
    B, Hk = _spread(rng, 1, 8), rng.choice([1, 2, 3, 4, 8])
    H = Hk * rng.choice([1, 1, 2, 3, 4])
    if op in ("forward", "backward", "step"):
        c = dict(op=op, B=B, H=H, Hk=Hk, T=1, d=d, dtype=rng.choice(["bf16", "bf16", "fp32"]), ragged=False, gated=op != "backward" and rng.random() < 0.3)
        if op == "step":
            c["B"] = _spread(rng, 1, 64)
            return c
        c["ragged"] = rng.random() < 0.4
        most = 8 * 16 * 4096 * 64 * 64 // (B * H * d * d)
        c["T"] = _spread(rng, 2, max(2, min(8192, most)))
        return c
    S = _spread(rng, 40, 9000)
    T = 1 if rng.random() < 0.3 else _spread(rng, 1, min(S, 2000))
    if T == 1 and op == "attend":
        B = _spread(rng, 1, 32)
    c = dict(op=op, B=B, H=H, Hk=Hk, T=T, d=d, dtype=rng.choice(["bf16", "e4m3"]), S=S, page=rng.choice([16, 32, 64, 128]), ragged=rng.random() < 0.4)
    if op == "cache":
        c["H"] = Hk
        return c
    while c["B"] * H * T * S > 2 * 16 * 2048 * 9000:
        c["B"] = max(1, c["B"] // 2)
        T = c["T"] = max(1, T // 2)
    c["window"] = rng.choice([0, 0, _spread(rng, 16, 2048)])
    c["sinks"] = rng.choice([0, 16]) if c["window"] else 0
    return c


def _counts(c):
    """Valid tokens of each sequence's T: all, or down to half of them in a padded batch."""
    return [c["T"] - (b * c["T"]) // (2 * c["B"]) if c["ragged"] else c["T"] for b in range(c["B"])]


def _starts(c):
    """Tokens that each sequence's cache holds before the chunk: S - T for the first, fewer for the others."""
    return [(c["S"] - c["T"]) - (b * (c["S"] - c["T"])) // (2 * c["B"]) for b in range(c["B"])]


def _quantise(x):
    """x [.., d] float32 -> e4m3 values and their power-of-two scales [..]."""
    m, e = torch.frexp(x.abs().amax(-1))  # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    scale = torch.ldexp(torch.ones_like(m), torch.where(m > 0, e, torch.zeros_like(e)))
    return (x / scale[..., None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    c, dev = case, "cuda"
    G = torch.Generator(device=dev).manual_seed(seed)
    tok = torch.float32 if c["dtype"] == "fp32" else torch.bfloat16
    normal = lambda *s: torch.randn(*s, generator=G, device=dev)  # noqa: E731
    unit = lambda x: x / x.square().sum(-1, keepdim=True).sqrt()  # noqa: E731
    s = {"case": c}
    B, H, Hk, T, d = (c[n] for n in ("B", "H", "Hk", "T", "d"))
    if c["op"] in ("forward", "backward", "step"):
        s["k"], s["q"] = (unit(normal(B, Hk, T, d)).to(tok) for _ in range(2))
        s["v"] = normal(B, H, T, d).to(tok)
        s["g"] = torch.log1p(-0.05 * torch.rand(B, H, T, generator=G, device=dev))
        s["beta"] = torch.sigmoid(normal(B, H, T))
        s["W"] = normal(B, H, d, d) * 0.3
        s["lengths"] = torch.tensor(_counts(c), dtype=torch.int32, device=dev) if c["ragged"] else None
        s["attn"] = normal(B, H, T, d).to(tok) if c["gated"] else None
        if c["op"] == "backward":
            s["dy"], s["dW"] = normal(B, H, T, d).to(tok), normal(B, H, d, d) * 0.3
        if c["op"] == "step":
            for n in ("k", "q", "v", "g", "beta", "attn"):
                s[n] = s[n][:, :, 0].contiguous() if s[n] is not None else None
        if own:
            from titans_long_term_b200 import DeltaMemory
            s["memory"] = DeltaMemory(d, c["dtype"], B, H, k_heads=Hk)
        return s
    page, most = c["page"], -(-c["S"] // c["page"])
    pages = B * most + 3
    s["table"] = torch.randperm(pages, generator=G, device=dev)[: B * most].to(torch.int32).reshape(B, most)
    s["starts"] = torch.tensor(_starts(c), dtype=torch.int32, device=dev)
    s["counts"] = torch.tensor(_counts(c), dtype=torch.int32, device=dev) if c["ragged"] else None
    s["pages"] = {}
    for n in ("k", "v"):
        x = normal(pages, Hk, page, d)
        if c["dtype"] == "e4m3":
            s["pages"][n], s["pages"][n + "_scale"] = _quantise(x)
        else:
            s["pages"][n] = x.to(torch.bfloat16)
    if c["op"] == "cache":
        s["k"], s["v"] = (normal(B, Hk, T, d).to(torch.bfloat16) for _ in range(2))
    else:
        s["q"] = normal(B, H, T, d).to(torch.bfloat16)
    if own:
        from titans_long_term_b200 import PagedCache
        s["memory"] = PagedCache(d, c["dtype"], B, H, kv_heads=Hk, page=page, num_pages=pages, max_pages=most)
    return s


def run(s):
    c = s["case"]
    if own:
        m = s["memory"]
        if c["op"] == "forward":
            y = m.forward(s["k"], s["q"], s["v"], s["g"], s["beta"], {"W": s["W"]}, lengths=s["lengths"], attn=s["attn"])
            return {"y": y, "W": s["W"]}
        if c["op"] == "step":
            return {"y": m.step(s["k"], s["q"], s["v"], s["g"], s["beta"], {"W": s["W"]}, attn=s["attn"]), "W": s["W"]}
        if c["op"] == "backward":
            return m.backward(s["k"], s["q"], s["v"], s["g"], s["beta"], {"W": s["W"]}, s["dy"], dstate={"W": s["dW"]}, lengths=s["lengths"])
        if c["op"] == "cache":
            m.append(s["k"], s["v"], s["pages"], s["table"], s["starts"], counts=s["counts"])
            k, v = m.read(s["pages"], s["table"], s["starts"], c["T"], counts=s["counts"])
            return {"k": k, "v": v}
        return {"o": m.attend(s["q"], s["pages"], s["table"], s["starts"], counts=s["counts"], window=c["window"], sinks=c["sinks"])}
    return {"forward": _forward, "step": _step, "backward": _backward, "cache": _cache, "attend": _attend}[c["op"]](s)


# ---------------------------------------------------------------- plain forms of the gated delta rule


def _valid(lengths, B, T, like):
    """[B, 1, T] truth values: the tokens that count."""
    if lengths is None:
        return torch.ones(B, 1, T, dtype=torch.bool, device=like.device)
    return torch.arange(T, device=like.device)[None, None] < lengths[:, None, None]


def _chunks(s, names):
    """Tokens as float32 [B, H, chunks, CHUNK, d], the shared heads repeated and the last chunk padded; a token
    that does not count neither decays (g = 0) nor writes (beta = 0)."""
    c = s["case"]
    B, H, T, d = s["v"].shape
    live = _valid(s["lengths"], B, T, s["v"])
    n = -(-T // CHUNK)
    out = {}
    for name in names:
        x = s[name].float()
        if name in ("k", "q"):
            x = x.repeat_interleave(H // c["Hk"], dim=1)
        x = torch.where(live if x.dim() == 3 else live[..., None], x, torch.zeros((), device=x.device))
        full = x.new_zeros(B, H, n * CHUNK, *x.shape[3:])
        full[:, :, :T] = x
        out[name] = full.reshape(B, H, n, CHUNK, *x.shape[3:])
    return out


def _within(x):
    """What a chunk's tokens need of one another: the cumulative decays and the inverse of I + A. The writes e
    of a chunk solve (I + A) e = beta (v - decay K W^T), A_ij = beta_i (decay from j to i) k_i.k_j for j < i."""
    G = x["g"].double().cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=G.device).tril()
    D = torch.where(low, (G[..., :, None] - G[..., None, :]).clamp(max=0).exp(), torch.zeros((), dtype=G.dtype, device=G.device)).float()
    A = (x["beta"][..., None] * D * (x["k"] @ x["k"].mT)).tril(-1)
    inv = torch.eye(CHUNK, device=G.device).expand_as(A).clone()
    for i in range(1, CHUNK):  # forward substitution, a row at a time
        inv[..., i, :i] = -(A[..., i, None, :i] @ inv[..., :i, :i])[..., 0, :]
    return G.exp().float(), (G[..., -1:] - G).exp().float(), D, inv


def _forward(s):
    c = s["case"]
    B, H, T, d = s["v"].shape
    x = _chunks(s, ("k", "q", "v", "g", "beta"))
    decay, rest, D, inv = _within(x)
    P = D * (x["q"] @ x["k"].mT)
    W, y = s["W"], torch.empty_like(x["v"])
    for n in range(y.shape[2]):  # the state goes from chunk to chunk
        k, q, v, a = x["k"][:, :, n], x["q"][:, :, n], x["v"][:, :, n], decay[:, :, n, :, None]
        e = inv[:, :, n] @ (x["beta"][:, :, n, :, None] * (v - a * (k @ W.mT)))
        y[:, :, n] = a * (q @ W.mT) + P[:, :, n] @ e
        W = decay[:, :, n, -1, None, None] * W + (rest[:, :, n, :, None] * e).mT @ k
    s["W"].copy_(W)
    y = y.reshape(B, H, -1, d)[:, :, :T]
    if s["attn"] is not None:
        y = s["attn"].float() * torch.sigmoid(y)
    y = torch.where(_valid(s["lengths"], B, T, y)[..., None], y, torch.zeros((), device=y.device))
    return {"y": y.to(s["v"].dtype), "W": s["W"]}


def _step(s):
    c = s["case"]
    k, q = (s[n].float().repeat_interleave(c["H"] // c["Hk"], dim=1) for n in ("k", "q"))
    A = s["g"].exp()[..., None, None] * s["W"]
    e = s["beta"][..., None] * (s["v"].float() - (A @ k[..., None])[..., 0])
    s["W"].copy_(A + e[..., None] * k[..., None, :])
    y = (s["W"] @ q[..., None])[..., 0]
    if s["attn"] is not None:
        y = s["attn"].float() * torch.sigmoid(y)
    return {"y": y.to(s["v"].dtype), "W": s["W"]}


def _backward(s):
    """Gradients of <dy, y> + <dW, W_T>, chunk by chunk: the forward's states, then the adjoint from the end."""
    c = s["case"]
    B, H, T, d = s["v"].shape
    x = _chunks(s, ("k", "q", "v", "g", "beta", "dy"))
    decay, rest, D, inv = _within(x)
    kk, qk = x["k"] @ x["k"].mT, x["q"] @ x["k"].mT
    W, states, N = s["W"], [], x["v"].shape[2]
    for n in range(N):
        k, b, a = x["k"][:, :, n], x["beta"][:, :, n, :, None], decay[:, :, n, :, None]
        states.append(W)
        e = inv[:, :, n] @ (b * (x["v"][:, :, n] - a * (k @ W.mT)))
        W = decay[:, :, n, -1, None, None] * W + (rest[:, :, n, :, None] * e).mT @ k
    out = {n: torch.empty_like(x["v"]) for n in ("k", "q", "v")}
    dG, dbeta, dW = torch.empty_like(x["g"]), torch.empty_like(x["g"]), s["dW"]
    for n in reversed(range(N)):
        k, q, v, dy = (x[m][:, :, n] for m in ("k", "q", "v", "dy"))
        b, a, l = x["beta"][:, :, n, :, None], decay[:, :, n, :, None], rest[:, :, n, :, None]
        W, Dn, ti = states[n], D[:, :, n], inv[:, :, n]
        m0 = a * (k @ W.mT)
        e = ti @ (b * (v - m0))
        P = Dn * qk[:, :, n]
        far = k @ dW.mT  # the adjoint of the final state, seen by each write
        de = P.mT @ dy + l * far
        dr = ti.mT @ de
        dP = (dy @ e.mT) * Dn
        dA = -(dr @ e.mT).tril(-1) * Dn
        dAb = dA * b
        out["v"][:, :, n] = b * dr
        out["q"][:, :, n] = a * (dy @ W) + dP @ k
        out["k"][:, :, n] = -(a * b * dr) @ W + l * (e @ dW) + dP.mT @ q + (dAb + dAb.mT) @ k
        dbeta[:, :, n] = (dr * (v - m0)).sum(-1) + (dA * kk[:, :, n]).sum(-1)
        pair = dP * qk[:, :, n] + dAb * kk[:, :, n]
        own_state = (l * e * far).sum(-1)
        dg = pair.sum(-1) - pair.sum(-2) - (b * dr * m0).sum(-1) + (dy * a * (q @ W.mT)).sum(-1) - own_state
        last = decay[:, :, n, -1, None, None]
        dg[..., -1] += own_state.sum(-1) + (last * dW * W).sum((-1, -2))
        dG[:, :, n] = dg
        dW = last * dW + dy.mT @ (a * q) - (a * b * dr).mT @ k
    dg = dG.double().flip(-1).cumsum(-1).flip(-1).float()
    live = _valid(s["lengths"], B, T, s["v"])
    cut = lambda t: t.reshape(B, H, -1, *t.shape[4:])[:, :, :T]  # noqa: E731
    only = lambda t: torch.where(live if t.dim() == 3 else live[..., None], t, torch.zeros((), device=t.device))  # noqa: E731
    r = {n: only(cut(out[n])) for n in ("k", "q", "v")}
    for n in ("k", "q"):
        r[n] = r[n].reshape(B, c["Hk"], H // c["Hk"], T, d).sum(2)
    r = {n: t.to(s["v"].dtype) for n, t in r.items()}
    return r | {"g": only(cut(dg)), "beta": only(cut(dbeta)), "W": dW}


# ---------------------------------------------------------------- plain forms of the paged cache


def _places(s, positions):
    """(page, slot) of positions [B, n] of each sequence, and whether the table has them."""
    size, table = s["case"]["page"], s["table"]
    index = positions.long() // size
    there = (positions >= 0) & (index < table.shape[1])
    return table.gather(1, index.clamp(0, table.shape[1] - 1)).long(), positions.long() % size, there


def _rows(s, n, positions, dtype):
    """Cached k or v of positions [B, n] -> [B, Hk, n, d] in dtype."""
    page, slot, _ = _places(s, positions)
    x = s["pages"][n].view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn).to(dtype) if s["case"]["dtype"] == "e4m3" else s["pages"][n][page, :, slot].to(dtype)
    if s["case"]["dtype"] == "e4m3":
        x = x * s["pages"][n + "_scale"][page, :, slot].to(dtype)[..., None]
    return x.transpose(1, 2)


def _cache(s):
    c = s["case"]
    t = torch.arange(c["T"], device=s["table"].device)
    live = _valid(s["counts"], c["B"], c["T"], s["table"])[:, 0]
    positions = s["starts"][:, None] + t[None]
    page, slot, there = _places(s, positions)
    page, slot = page[live & there], slot[live & there]
    for n in ("k", "v"):
        x = s[n].transpose(1, 2)[live & there].float()
        if c["dtype"] == "e4m3":
            x, scale = _quantise(x)
            s["pages"][n].view(torch.uint8)[page, :, slot] = x.view(torch.uint8)
            s["pages"][n + "_scale"][page, :, slot] = scale
        else:
            s["pages"][n][page, :, slot] = x.to(torch.bfloat16)
    zero = torch.zeros((), device=live.device)
    return {n: torch.where(live[:, None, :, None], _rows(s, n, positions, torch.float32), zero).to(torch.bfloat16) for n in ("k", "v")}


def _visible(c, at, keys):
    """Whether the query at a position sees a key: [.., queries, keys]."""
    p, j = at[..., :, None], keys
    seen = j <= p
    if c["window"]:
        seen = seen & ((j > p - c["window"]) | (j < c["sinks"]))
    return seen


def _attend(s):
    c = s["case"]
    dev, B, H = s["q"].device, c["B"], c["H"]
    t = torch.arange(c["T"], device=dev)
    keys = torch.arange(c["S"], device=dev)
    at = s["starts"][:, None] + t[None]
    seen = (_visible(c, at, keys) & _valid(s["counts"], B, c["T"], s["q"])[:, 0, :, None])[:, None]
    k, v = (_rows(s, n, keys[None].expand(B, -1), torch.float32).repeat_interleave(H // c["Hk"], dim=1) for n in ("k", "v"))
    z = (s["q"].float() @ k.mT) * (c["d"] ** -0.5)
    z = z.masked_fill(~seen, float("-inf"))
    top = z.amax(-1, keepdim=True).clamp(min=torch.finfo(z.dtype).min)
    p = (z - top).exp()
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total > 0, total, torch.ones_like(total))
    return {"o": o.to(torch.bfloat16)}


# ---------------------------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    return {"forward": _exact_forward, "step": _exact_forward, "backward": _exact_backward, "cache": _exact_cache, "attend": _exact_attend}[case["op"]](s)


def _tokens64(s):
    """Per-token double tensors [B, H, T, ..] and the number of tokens of each sequence."""
    c = s["case"]
    step = c["op"] == "step"
    get = lambda n: (s[n][:, :, None] if step else s[n]).double()  # noqa: E731
    x = {n: get(n) for n in ("k", "q", "v", "g", "beta")}
    for n in ("k", "q"):
        x[n] = x[n][:, torch.arange(c["H"], device="cuda") // (c["H"] // c["Hk"])]
    return x, torch.tensor(_counts(c), device="cuda")


def _advance(W, x, t, live):
    """W_{t-1} -> (W_t, e_t, decayed W_{t-1}); the sequences that have ended keep theirs."""
    k, v = x["k"][:, :, t], x["v"][:, :, t]
    A = W * torch.exp(x["g"][:, :, t])[..., None, None]
    e = (v - torch.einsum("bhij,bhj->bhi", A, k)) * x["beta"][:, :, t, None]
    new = A + torch.einsum("bhi,bhj->bhij", e, k)
    return torch.where(live[:, None, None, None], new, W), e, A


def _exact_forward(s):
    c = s["case"]
    x, n = _tokens64(s)
    W, ys = s["W"].double(), []
    for t in range(c["T"]):
        live = t < n
        W, _, _ = _advance(W, x, t, live)
        ys.append(torch.einsum("bhij,bhj->bhi", W, x["q"][:, :, t]) * live[:, None, None])
    y = torch.stack(ys, 2)
    if c["gated"]:
        attn = s["attn"][:, :, None] if c["op"] == "step" else s["attn"]
        y = attn.double() / (1 + torch.exp(-y)) * (torch.arange(c["T"], device="cuda") < n[:, None])[:, None, :, None]
    return {"y": y[:, :, 0] if c["op"] == "step" else y, "W": W}


def _exact_backward(s):
    c = s["case"]
    if c["T"] > 9000:
        return None
    x, n = _tokens64(s)
    dy, block = s["dy"].double(), 64
    W, kept = s["W"].double(), []
    for t in range(c["T"]):
        if t % block == 0:
            kept.append(W)
        W, _, _ = _advance(W, x, t, t < n)
    r = {m: torch.zeros_like(x[m]) for m in x}
    dW = s["dW"].double()
    for at in reversed(range(0, c["T"], block)):
        before, W = [], kept[at // block]
        for t in range(at, min(at + block, c["T"])):
            before.append(W)
            W, _, _ = _advance(W, x, t, t < n)
        for t in reversed(range(at, min(at + block, c["T"]))):
            live = (t < n)[:, None, None]
            W0 = before[t - at]
            W1, e, A = _advance(W0, x, t, t < n)
            k, q, b, u = x["k"][:, :, t], x["q"][:, :, t], x["beta"][:, :, t, None], dy[:, :, t]
            full = dW + torch.einsum("bhi,bhj->bhij", u, q)
            de = torch.einsum("bhij,bhj->bhi", full, k)
            fall = full - torch.einsum("bhi,bhj->bhij", b * de, k)
            r["q"][:, :, t] = torch.einsum("bhij,bhi->bhj", W1, u) * live
            r["k"][:, :, t] = (torch.einsum("bhij,bhi->bhj", full, e) - torch.einsum("bhij,bhi->bhj", A, b * de)) * live
            r["v"][:, :, t] = b * de * live
            r["beta"][:, :, t] = (de * (x["v"][:, :, t] - torch.einsum("bhij,bhj->bhi", A, k))).sum(-1) * live[..., 0]
            r["g"][:, :, t] = (fall * A).sum((-1, -2)) * live[..., 0]
            dW = torch.where(live[..., None], fall * torch.exp(x["g"][:, :, t])[..., None, None], dW)
    for m in ("k", "q"):
        r[m] = r[m].reshape(c["B"], c["Hk"], -1, c["T"], c["d"]).sum(2)
    return r | {"W": dW}


def _exact_cache(s):
    c = s["case"]
    out = {}
    live = torch.arange(c["T"], device="cuda")[None] < torch.tensor(_counts(c), device="cuda")[:, None]
    for n in ("k", "v"):
        x = s[n].double()
        if c["dtype"] == "e4m3":
            scale = torch.exp2(torch.ceil(torch.log2(x.abs().amax(-1, keepdim=True) / 448)))
            y = x / scale
            ulp = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0**-6))) - 3)  # 3 bits after the leading one
            x = torch.round(y / ulp) * ulp * scale
        out[n] = x * live[:, None, :, None]
    return out


def _exact_attend(s):
    c = s["case"]
    B, H, T, d = s["q"].shape
    out = torch.zeros(B, H, T, d, dtype=torch.float64, device="cuda")
    for b, (start, count) in enumerate(zip(_starts(c), _counts(c))):
        keys = torch.arange(start + count, device="cuda")
        at = torch.arange(start, start + count, device="cuda")
        seen = _visible(c, at, keys)
        one = {**s, "table": s["table"][b : b + 1]}
        k, v = (_rows(one, n, keys[None], torch.float64)[0] for n in ("k", "v"))
        for h in range(H):
            z = s["q"][b, h, :count].double() @ k[h // (H // c["Hk"])].mT / d**0.5
            p = torch.where(seen, torch.exp(z - z.masked_fill(~seen, -1e300).amax(-1, keepdim=True)), torch.zeros((), dtype=z.dtype, device="cuda"))
            out[b, h, :count] = (p @ v[h // (H // c["Hk"])]) / p.sum(-1, keepdim=True)
    return {"o": out}


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    c = case
    H, Hk, d, n = c["H"], c["Hk"], c["d"], sum(_counts(c))
    if c["op"] in ("forward", "step", "backward"):
        e = 4 if c["dtype"] == "fp32" else 2
        state = 4 * c["B"] * H * d * d
        if c["op"] == "backward":  # k, q and their gradients; v, dy, dv; g, beta and theirs; W, dW and the gradient of W
            return {"bytes": n * d * e * (4 * Hk + 3 * H) + 16 * n * H + 3 * state, "flops": 18 * n * H * d * d}
        return {"bytes": n * d * e * (2 * Hk + (3 if c["gated"] else 2) * H) + 8 * n * H + 2 * state, "flops": 6 * n * H * d * d}
    row = (d + 4) if c["dtype"] == "e4m3" else 2 * d  # one cached k or v of one token and head
    if c["op"] == "cache":  # k, v read and written to the cache, read back and written out
        return {"bytes": 2 * n * Hk * (2 * d + row + row + 2 * d), "flops": 0}
    pairs = keys = 0
    for start, count in zip(_starts(c), _counts(c)):
        w, k = c["window"], c["sinks"]
        for p in (start, start + count - 1):  # the visible keys grow evenly from the first query to the last
            pairs += count / 2 * (p + 1 if not w else min(p + 1, w) + max(0, min(k, p + 1 - w)))
        keys += start + count if not w else min(start + count, w + count - 1 + k)
    return {"bytes": 4 * n * H * d + 2 * keys * Hk * row, "flops": 4 * pairs * H * d}
