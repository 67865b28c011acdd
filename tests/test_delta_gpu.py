"""The gated delta rule on the GPU against the recurrence in 64 bits (delta_ref)."""
import gc

import pytest
import torch

import delta_ref
from delta_ref import assert_close
from titans_long_term_b200 import DeltaMemory

pytestmark = pytest.mark.gpu


def make(B, H, Hk, T, d, mode, **kw):
    x = delta_ref.inputs(B, H, Hk, T, d, mode, device="cuda", **kw)
    return DeltaMemory(d, mode, B, H, k_heads=Hk), x


def call(m, x, gated=False, lengths=True, **kw):
    W = x["W"].clone()
    y = m.forward(x["k"], x["q"], x["v"], x["g"], x["beta"], {"W": W}, lengths=x["lengths"] if lengths else None,
                  attn=x["attn"] if gated else None, **kw)
    return y, W


@pytest.mark.parametrize("mode", ["bf16", "fp32"])
@pytest.mark.parametrize("B,H,Hk,T,d", [
    (1, 1, 1, 1, 64), (2, 4, 4, 2, 128), (1, 2, 2, 15, 64), (1, 2, 1, 31, 128), (2, 3, 1, 63, 64), (1, 4, 2, 64, 128),
    (1, 2, 2, 65, 64), (2, 2, 1, 130, 128), (3, 6, 2, 257, 64), (1, 1, 1, 700, 128), (5, 4, 4, 333, 64)])
def test_forward(B, H, Hk, T, d, mode):
    m, x = make(B, H, Hk, T, d, mode, seed=T)
    y, W = call(m, x)
    ry, rW = delta_ref.forward(x)
    assert_close("y", y, ry, mode)
    assert_close("W", W, rW, "fp32")


@pytest.mark.parametrize("mode", ["bf16", "fp32"])
@pytest.mark.parametrize("B,H,Hk,T,d", [(5, 2, 1, 3, 64), (5, 2, 2, 150, 128), (5, 3, 3, 200, 64)])
def test_forward_ragged_gated(B, H, Hk, T, d, mode):
    """Lengths of 0, 1, T / 2, T - 1 and T; what stands behind them, NaN too, reaches nothing, and y = 0 there."""
    m, x = make(B, H, Hk, T, d, mode, seed=T, ragged=True)
    ry, rW = delta_ref.forward(x, gated=True)
    for b, n in enumerate(x["lengths"].tolist()):
        for name in ("k", "q", "v", "g", "beta", "attn"):
            x[name][b, :, n:] = float("nan")
    y, W = call(m, x, gated=True)
    assert_close("y", y, ry, mode)
    assert_close("W", W, rW, "fp32")
    for b, n in enumerate(x["lengths"].tolist()):
        assert (y[b, :, n:] == 0).all()
    assert torch.equal(W[1], x["W"][1])  # length 0: untouched


@pytest.mark.parametrize("T", [7, 90, 300])
@pytest.mark.parametrize("mode", ["bf16", "fp32"])
def test_forward_resets_and_silent_tokens(T, mode):
    """g = -inf forgets everything, beta = 0 writes nothing."""
    m, x = make(2, 2, 2, T, 64, mode, seed=T, reset=True)
    y, W = call(m, x)
    ry, rW = delta_ref.forward(x)
    assert_close("y", y, ry, mode)
    assert_close("W", W, rW, "fp32")


@pytest.mark.parametrize("change", ["large values", "small values", "small keys", "strong decay", "same key"])
def test_forward_ranges(change):
    m, x = make(1, 2, 2, 200, 64, "fp32", seed=5)
    if change == "large values":
        x["v"] *= 1e12
    elif change == "small values":
        x["v"] *= 1e-12
        x["W"] *= 1e-12
    elif change == "small keys":
        x["k"] *= 1e-5
    elif change == "strong decay":
        x["g"] *= 400
    else:  # every token overwrites the same direction
        x["k"][:] = x["k"][:, :, :1]
        x["beta"][:] = 1
    y, W = call(m, x)
    ry, rW = delta_ref.forward(x)
    assert_close("y", y, ry, "fp32")
    assert_close("W", W, rW, "fp32")


def test_forward_in_two_calls():
    """A stream cut at any token goes on from its state."""
    m, x = make(2, 2, 2, 301, 64, "fp32", seed=1)
    ry, rW = delta_ref.forward(x)
    state = {"W": x["W"].clone()}
    ys = []
    for lo, hi in ((0, 77), (77, 78), (78, 301)):
        z = {n: x[n][:, :, lo:hi].contiguous() for n in ("k", "q", "v", "g", "beta")}
        ys.append(m.forward(*z.values(), state))
    assert_close("y", torch.cat(ys, 2), ry, "fp32")
    assert_close("W", state["W"], rW, "fp32")


@pytest.mark.parametrize("mode", ["bf16", "fp32"])
@pytest.mark.parametrize("B,H,Hk,d", [(1, 1, 1, 64), (3, 4, 2, 128), (2, 5, 5, 64)])
def test_step(B, H, Hk, d, mode):
    m, x = make(B, H, Hk, 3, d, mode, seed=d + B)
    ry, rW = delta_ref.forward(x)
    go, _ = delta_ref.forward(x, gated=True)
    state = {"W": x["W"].clone()}
    for t in range(3):
        z = {n: x[n][:, :, t].contiguous() for n in ("k", "q", "v", "g", "beta", "attn")}
        attn = z.pop("attn") if t == 1 else (z.pop("attn"), None)[1]
        y = m.step(*z.values(), state, attn=attn)
        assert_close("y", y[:, :, None], (go if t == 1 else ry)[:, :, t, None], mode)
    assert_close("W", state["W"], rW, "fp32")


def test_other_stream_and_outputs():
    """A call on its own stream, with its own output, equals the plain one bit for bit; so does one replayed from
    a graph with new inputs in the captured tensors."""
    m, x = make(2, 4, 2, 150, 64, "bf16", seed=9)
    y0, W0 = call(m, x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y1 = torch.full_like(x["v"], float("nan"))
    _, W1 = call(m, x, y=y1, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(y0, y1) and torch.equal(W0, W1)
    z = {n: t.clone() for n, t in x.items()}
    W = {"W": z["W"].clone()}
    gc.collect()  # handles of other memories that are still waiting to be collected would end the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2 = m.forward(z["k"], z["q"], z["v"], z["g"], z["beta"], W, lengths=z["lengths"])
    other = delta_ref.inputs(2, 4, 2, 150, 64, "bf16", device="cuda", seed=10)
    for new in (other, x):
        for n in z:
            z[n].copy_(new[n])
        W["W"].copy_(new["W"])
        graph.replay()
        ye, We = call(m, new)
        assert torch.equal(y2, ye) and torch.equal(W["W"], We)


def test_binding_refuses_tensors():
    m, x = make(1, 2, 1, 8, 64, "bf16")
    state = {"W": x["W"]}
    good = [x[n] for n in ("k", "q", "v", "g", "beta")]
    for i, bad in ((0, x["k"].float()), (0, x["v"]), (1, x["q"].cpu()), (2, x["v"].transpose(-1, -2)), (3, x["g"].double()),
                   (4, x["beta"][:, :1]), (2, x["v"][:, :, ::2])):
        args = list(good)
        args[i] = bad
        with pytest.raises(ValueError):
            m.forward(*args, state)
    with pytest.raises(ValueError, match="lengths"):
        m.forward(*good, state, lengths=torch.tensor([3], device="cuda"))
    with pytest.raises(ValueError, match="W"):
        m.forward(*good, {"W": x["W"].half()})


def grads(m, x, with_dW=True, **kw):
    W = x["W"].clone()
    out = m.backward(x["k"], x["q"], x["v"], x["g"], x["beta"], {"W": W}, x["dy"],
                     dstate={"W": x["dW"]} if with_dW else None, lengths=x["lengths"], **kw)
    assert torch.equal(W, x["W"])  # read only
    return out


def check_grads(out, want, mode):
    for n in ("k", "q", "v"):
        assert_close(n, out[n], want[n], mode)
    for n in ("g", "beta", "W"):
        assert_close(n, out[n], want[n], "fp32")


@pytest.mark.parametrize("mode", ["bf16", "fp32"])
@pytest.mark.parametrize("B,H,Hk,T,d", [
    (1, 1, 1, 1, 64), (2, 2, 2, 5, 128), (1, 2, 1, 64, 64), (1, 2, 1, 65, 128), (2, 6, 2, 130, 64), (1, 3, 3, 200, 128),
    (1, 4, 1, 449, 64), (5, 4, 2, 128, 128)])
def test_backward(B, H, Hk, T, d, mode):
    m, x = make(B, H, Hk, T, d, mode, seed=T)
    check_grads(grads(m, x), delta_ref.backward(x), mode)


@pytest.mark.parametrize("mode", ["bf16", "fp32"])
@pytest.mark.parametrize("B,H,Hk,T,d", [(5, 2, 1, 3, 64), (5, 4, 2, 200, 64), (5, 2, 2, 140, 128)])
def test_backward_ragged(B, H, Hk, T, d, mode):
    """Gradients behind the lengths are zero, and nothing there is read."""
    m, x = make(B, H, Hk, T, d, mode, seed=T, ragged=True)
    want = delta_ref.backward(x)
    for b, n in enumerate(x["lengths"].tolist()):
        for name in ("k", "q", "v", "g", "beta", "dy"):
            x[name][b, :, n:] = float("nan")
    out = grads(m, x)
    check_grads(out, want, mode)
    for b, n in enumerate(x["lengths"].tolist()):
        for name in ("k", "q", "v", "g", "beta"):
            assert (out[name][b, :, n:] == 0).all()
    assert torch.equal(out["W"][1], x["dW"][1])  # length 0


@pytest.mark.parametrize("T", [20, 150])
def test_backward_resets_and_silent_tokens(T):
    """beta = 0 has its gradient all the same; nothing flows through a decay of 0 (its g gets none)."""
    m, x = make(2, 2, 2, T, 64, "fp32", seed=T, reset=True)
    want = delta_ref.backward(x)
    check_grads(grads(m, x), want, "fp32")


def test_backward_without_state_gradient():
    m, x = make(2, 2, 2, 100, 64, "fp32", seed=8)
    x["dW"].zero_()
    check_grads(grads(m, x, with_dW=False), delta_ref.backward(x), "fp32")


def test_backward_against_differences():
    """A step along a random direction changes the forward's value by its product with the gradient: central differences
    of the fp32 forward, whose value is off by about 2^-22 of |dy| |y|, over a step of 2^-7."""
    m, x = make(1, 2, 1, 96, 64, "fp32", seed=12)

    def value(z):
        y, W = call(m, z)
        return float((y.double() * x["dy"].double()).sum() + (W.double() * x["dW"].double()).sum())

    out = grads(m, x)
    G = torch.Generator().manual_seed(1)
    h = 2.0**-7
    y, _ = call(m, x)
    noise = 2**-21 * float(x["dy"].norm() * y.norm() + x["dW"].norm() * x["W"].norm()) / h
    for n in ("k", "q", "v", "g", "beta", "W"):
        way = torch.randn(x[n].shape, generator=G).cuda()
        way /= way.norm()
        d1 = (value({**x, n: x[n] + h * way}) - value({**x, n: x[n] - h * way})) / (2 * h)
        d2 = (value({**x, n: x[n] + 2 * h * way}) - value({**x, n: x[n] - 2 * h * way})) / (4 * h)
        change = (4 * d1 - d2) / 3  # the cubic term taken out
        assert abs(change - float((out[n].double() * way.double()).sum())) <= 4 * noise + abs(d1 - d2), n


def test_backward_repeats_and_captures():
    """The same call twice, on another stream and replayed from a graph: the same bits."""
    m, x = make(2, 4, 2, 150, 128, "bf16", seed=3)
    first, s = grads(m, x), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    second = grads(m, x, stream=s)
    torch.cuda.synchronize()
    gc.collect()  # handles of other memories that are still waiting to be collected would end the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = m.backward(x["k"], x["q"], x["v"], x["g"], x["beta"], {"W": x["W"]}, x["dy"],
                           dstate={"W": x["dW"]}, lengths=x["lengths"])
    graph.replay()
    torch.cuda.synchronize()
    for n in first:
        assert torch.equal(first[n], second[n]) and torch.equal(first[n], third[n]), n


@pytest.mark.parametrize("mode", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [24, 25])
def test_forward_where_chunks_begin(T, mode):
    """The longest call that goes token by token, and the shortest one in chunks."""
    m, x = make(2, 4, 2, T, 128, mode, seed=T)
    y, W = call(m, x)
    ry, rW = delta_ref.forward(x)
    assert_close("y", y, ry, mode)
    assert_close("W", W, rW, "fp32")
