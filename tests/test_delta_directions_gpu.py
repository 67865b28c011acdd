"""Each gradient of the gated delta rule against the change of the 64-bit forward along that very gradient."""
import pytest
import torch

import delta_ref
from titans_long_term_b200 import DeltaMemory

pytestmark = pytest.mark.gpu


def value(x):
    y, W = delta_ref.forward(x)
    return float((y * x["dy"]).sum() + (W * x["dW"]).sum())


@pytest.mark.parametrize("name", ["k", "q", "v", "g", "beta", "W"])
@pytest.mark.parametrize("B,H,Hk,T,d", [(1, 2, 1, 96, 64), (2, 2, 2, 20, 128), (3, 4, 2, 130, 64)])
def test_gradient_against_differences(B, H, Hk, T, d, name):
    """Along the gradient, scaled to length 1, the value changes by the gradient's norm. Central differences in 64 bits over
    h and 2 h, the cubic term taken out, are off by about 2^-53 |value| / h and h^4: with h = 2^-10 both are below 1e-9 of the
    change, so what is left is the gradient itself, off by NORM32 of its norm per unit."""
    x = delta_ref.inputs(B, H, Hk, T, d, "fp32", seed=T, device="cuda", ragged=B > 1)
    m = DeltaMemory(d, "fp32", B, H, k_heads=Hk)
    out = m.backward(x["k"], x["q"], x["v"], x["g"], x["beta"], {"W": x["W"]}, x["dy"], dstate={"W": x["dW"]},
                     lengths=x["lengths"])[name].double()
    way = out / out.norm()
    wide = {n: t.double() if t.is_floating_point() else t for n, t in x.items()}
    at = lambda s: value({**wide, name: wide[name] + s * way})  # noqa: E731
    h = 2.0**-10
    d1, d2 = (at(h) - at(-h)) / (2 * h), (at(2 * h) - at(-2 * h)) / (4 * h)
    change = (4 * d1 - d2) / 3
    bar = 2 * delta_ref.NORM32 * float(out.norm())
    assert abs(d1 - d2) <= 1e-3 * abs(change)  # the differences themselves have settled
    assert abs(change - float(out.norm())) <= bar
