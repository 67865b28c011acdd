"""The paged cache, its attention and the gated delta rule run together, as the layer of a serving loop and of a
training step uses them: each chunk of new tokens goes into the cache, attends over it, and the attention's output is gated by
the memory, whose state goes on from chunk to chunk and to single tokens."""
import pytest
import torch

import cache_ref
import delta_ref
from titans_long_term_b200 import DeltaMemory, Memory, PagedCache, new_state

pytestmark = pytest.mark.gpu

B, H, HKV, D = 3, 4, 2, 64


def stream(T, seed):
    x = delta_ref.inputs(B, H, HKV, T, D, "bf16", device="cuda", seed=seed)
    G = torch.Generator().manual_seed(seed)
    new = lambda heads: torch.randn(B, heads, T, D, generator=G).to(torch.bfloat16).cuda()  # noqa: E731
    return x, new(H), new(HKV), new(HKV)


def cut(t, lo, hi):
    return t[:, :, lo:hi].contiguous()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_serving_in_chunks_and_tokens(dtype):
    T = 230
    x, q, k, v = stream(T, 5)
    cache = PagedCache(D, dtype, B, H, kv_heads=HKV, page=16, num_pages=3 * 16, max_pages=16)
    memory = DeltaMemory(D, "bf16", B, H, k_heads=HKV)
    pages, state = cache.new_pages(), {"W": x["W"].clone()}
    table = torch.randperm(48, generator=torch.Generator().manual_seed(1)).to(torch.int32).reshape(B, 16).cuda()
    attns, outs = [], []
    for lo, hi in ((0, 100), (100, 107), (107, 228), (228, 229), (229, 230)):
        starts = torch.full((B,), lo, dtype=torch.int32, device="cuda")
        cache.append(cut(k, lo, hi), cut(v, lo, hi), pages, table, starts)
        attn = cache.attend(cut(q, lo, hi), pages, table, starts, window=150, sinks=4)
        z = [cut(x[n], lo, hi) for n in ("k", "q", "v", "g", "beta")]
        if hi - lo == 1:
            o = memory.step(*[t[:, :, 0].contiguous() for t in z], state, attn=attn[:, :, 0].contiguous())[:, :, None]
        else:
            o = memory.forward(*z, state, attn=attn)
        attns.append(attn)
        outs.append(o)
    cache.sync_status()
    attn, out = torch.cat(attns, 2), torch.cat(outs, 2)
    ck, cv = (k, v) if dtype == "bf16" else (cache_ref.quantise(k), cache_ref.quantise(v))
    want = cache_ref.attend(q, ck, cv, [0] * B, [T] * B, 150, 4)
    assert ((attn.double() - want).abs() / cache_ref.bar(want, cv)).max() <= 1
    x["attn"] = attn  # the gate is checked on the attention's own output
    ry, rW = delta_ref.forward(x, gated=True)
    delta_ref.assert_close("o", out, ry, "bf16")
    delta_ref.assert_close("W", state["W"], rW, "fp32")


def test_attention_gates_the_other_memories_too():
    T = 96
    x, q, k, v = stream(T, 7)
    cache = PagedCache(D, "bf16", B, H, kv_heads=HKV, page=32, num_pages=9, max_pages=3)
    pages, table = cache.new_pages(), torch.arange(9, dtype=torch.int32, device="cuda").reshape(B, 3)
    starts = torch.zeros(B, dtype=torch.int32, device="cuda")
    cache.append(k, v, pages, table, starts)
    attn = cache.attend(q, pages, table, starts)
    m = Memory(D, 4 * D, 32, "bf16", B, H)
    rep = lambda t: t.repeat_interleave(H // HKV, 1).contiguous()  # noqa: E731
    gate = torch.rand(B, H, T, device="cuda") * 0.01
    args = [rep(x["k"]), rep(x["q"]), x["v"], gate, gate, gate]
    y = m.forward(*args, new_state(B, H, D, 4 * D))
    o = m.forward_gated(*args[:6], attn, new_state(B, H, D, 4 * D))
    m.sync_status()
    # the gate is taken before y's rounding: half a step of y moves sigmoid(y) by 2^-9 |y| / 4 at most, and o is rounded once
    want = attn.double() * torch.sigmoid(y.double())
    bar = 2**-8 * want.abs() + 2**-10 * (attn.double() * y.double()).abs() + 1e-12
    assert ((o.double() - want).abs() <= bar).all()


def test_a_training_step():
    """Forward and backward of a stream in two segments equal those of the whole: the state's adjoint goes back through the cut."""
    T, at = 200, 77
    x, *_ = stream(T, 9)
    m = DeltaMemory(D, "bf16", B, H, k_heads=HKV)
    names = ("k", "q", "v", "g", "beta")
    parts = [[cut(x[n], lo, hi) for n in names] for lo, hi in ((0, at), (at, T))]
    dys = [cut(x["dy"], 0, at), cut(x["dy"], at, T)]
    middle = {"W": x["W"].clone()}
    m.forward(*parts[0], middle)
    late = m.backward(*parts[1], middle, dys[1], dstate={"W": x["dW"]})
    early = m.backward(*parts[0], {"W": x["W"]}, dys[0], dstate={"W": late["W"]})
    want = delta_ref.backward(x)
    for n in ("k", "q", "v"):
        delta_ref.assert_close(n, torch.cat([early[n], late[n]], 2), want[n], "bf16")
    for n in ("g", "beta"):
        delta_ref.assert_close(n, torch.cat([early[n], late[n]], 2), want[n], "fp32")
    delta_ref.assert_close("W", early["W"], want["W"], "fp32")


def test_two_streams_at_once():
    """Calls that overlap on the GPU share nothing: the same bits as one after the other."""
    T = 400
    xs = [stream(T, 20 + i) for i in range(2)]
    m = DeltaMemory(D, "bf16", B, H, k_heads=HKV)
    cache = PagedCache(D, "e4m3", B, H, kv_heads=HKV, page=64, num_pages=21, max_pages=7)
    table = torch.arange(21, dtype=torch.int32, device="cuda").reshape(B, 7)
    starts = torch.zeros(B, dtype=torch.int32, device="cuda")
    one = torch.full((B,), T - 1, dtype=torch.int32, device="cuda")

    def everything(i, s):
        x, q, k, v = xs[i]
        with torch.cuda.stream(s):
            pages, W = cache.new_pages(), x["W"].clone()
        cache.append(k, v, pages, table, starts, stream=s)
        o = cache.attend(q, pages, table, starts, stream=s)
        with torch.cuda.stream(s):
            last = q[:, :, -1:].contiguous()
        t = cache.attend(last, pages, table, one, stream=s)
        y = m.forward(x["k"], x["q"], x["v"], x["g"], x["beta"], {"W": W}, attn=o, stream=s)
        g = m.backward(x["k"], x["q"], x["v"], x["g"], x["beta"], {"W": x["W"]}, x["dy"], stream=s)
        return [o, t, y, W, *g.values()]

    alone = [everything(i, torch.cuda.current_stream()) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        both = [everything(i, streams[i]) for i in range(2)]
        torch.cuda.synchronize()
        for a, b in zip(alone, both):
            for p, q in zip(a, b):
                assert torch.equal(p, q)
