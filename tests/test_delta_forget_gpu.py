"""Markers for "forget all" other than -infinity, in calls of any length: the gated delta rule against 64 bits. A g below about
-104 is a decay of 0 in fp32."""
import pytest
import torch

import delta_ref
from delta_ref import assert_close
from titans_long_term_b200 import DeltaMemory

pytestmark = pytest.mark.gpu

LOWEST = torch.finfo(torch.float32).min


def marked(T, d, mode, where, marker, seed):
    x = delta_ref.inputs(2, 2, 1, T, d, mode, device="cuda", seed=seed)
    x["g"][:] = -0.05
    for t in where:
        if t < T:
            x["g"][:, :, t] = marker
    return DeltaMemory(d, mode, 2, 2, k_heads=1), x


@pytest.mark.parametrize("marker", [-float("inf"), LOWEST, -1e30, -1e15, -1e9, -1e4, -105.0, -103.0, -90.0])
@pytest.mark.parametrize("T,d,where", [
    (12, 64, [4]), (25, 64, [4, 9]), (64, 64, [20]), (64, 128, [21]), (70, 64, [21, 44]), (200, 64, [0, 63, 64, 65, 150, 151]),
    (200, 128, list(range(80, 140)))])
@pytest.mark.parametrize("mode", ["bf16", "fp32"])
def test_forgetting_tokens(T, d, where, marker, mode):
    m, x = marked(T, d, mode, where, marker, T)
    W = x["W"].clone()
    y = m.forward(x["k"], x["q"], x["v"], x["g"], x["beta"], {"W": W})
    ry, rW = delta_ref.forward(x)
    assert_close("y", y, ry, mode)
    assert_close("W", W, rW, "fp32")
    out = m.backward(x["k"], x["q"], x["v"], x["g"], x["beta"], {"W": x["W"]}, x["dy"], dstate={"W": x["dW"]})
    want = delta_ref.backward(x)
    for n in ("k", "q", "v"):
        assert_close(n, out[n], want[n], mode)
    for n in ("g", "beta", "W"):
        assert_close(n, out[n], want[n], "fp32")
