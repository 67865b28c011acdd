"""Nothing flows through a decay of 0: its g gets no gradient at all, wherever in a chunk it stands."""
import pytest
import torch

import delta_ref
from titans_long_term_b200 import DeltaMemory

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,share", [(1, 1.0), (63, 1.0), (64, 0.5), (65, 0.9), (130, 0.05), (200, 0.5), (200, 1.0)])
def test_no_gradient_of_forgetting_tokens(T, share, d, mode):
    x = delta_ref.inputs(2, 4, 2, T, d, mode, seed=T, device="cuda", ragged=True)
    G = torch.Generator().manual_seed(T)
    cut = (torch.rand(2, 4, T, generator=G) < share).cuda()
    x["g"][cut] = -float("inf")
    x["g"][:, 1][cut[:, 1]] = -1e6
    out = DeltaMemory(d, mode, 2, 4, k_heads=2).backward(
        x["k"], x["q"], x["v"], x["g"], x["beta"], {"W": x["W"]}, x["dy"], dstate={"W": x["dW"]}, lengths=x["lengths"])
    assert (out["g"][cut] == 0).all()
    want = delta_ref.backward(x)
    for n in ("k", "q", "v"):
        delta_ref.assert_close(n, out[n], want[n], mode)
    delta_ref.assert_close("W", out["W"], want["W"], "fp32")


@pytest.mark.parametrize("mode", ["bf16", "fp32"])
def test_gradients_before_a_forgetting_token(mode):
    """What comes from the token's own side of the cut: the gradients of 40 tokens before it equal those of a stream that ends there."""
    T, at = 64, 40
    x = delta_ref.inputs(2, 2, 2, T, 64, mode, seed=2, device="cuda")
    x["g"][:, :, at] = -float("inf")
    m = DeltaMemory(64, mode, 2, 2)
    names = ("k", "q", "v", "g", "beta")
    whole = m.backward(*[x[n] for n in names], {"W": x["W"]}, x["dy"], dstate={"W": x["dW"]})
    want = delta_ref.backward({**{n: x[n][:, :, :at] for n in (*names, "dy")}, "W": x["W"], "dW": torch.zeros_like(x["dW"]),
                               "lengths": x["lengths"].clamp(max=at)})
    for n in ("k", "q", "v"):
        delta_ref.assert_close(n, whole[n][:, :, :at], want[n], mode)
    for n in ("g", "beta"):
        delta_ref.assert_close(n, whole[n][:, :, :at], want[n], "fp32")
    delta_ref.assert_close("W", whole["W"], want["W"], "fp32")
