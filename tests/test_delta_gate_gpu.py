"""The gate of a large memory: attn * sigmoid(y) against 64 bits where y is far larger than what the gate tells apart."""
import pytest
import torch

import delta_ref
from titans_long_term_b200 import DeltaMemory

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode", ["bf16", "fp32"])
@pytest.mark.parametrize("size", [1.0, 30.0, 1000.0])
@pytest.mark.parametrize("B,H,Hk,T,d", [(2, 2, 2, 20, 64), (2, 4, 2, 200, 64), (3, 3, 1, 333, 128)])
def test_gate_of_large_values(B, H, Hk, T, d, size, mode):
    """Bar, value by value. y is off by NORM32 of its size (delta_ref), for which the largest |y| of the unit stands, so sigmoid(y)
    by at most a quarter of that and the output by |attn| times it; in mode bf16 the output is rounded once, by 2^-8 of itself at
    most, and in fp32 it comes from an exponential, a sum and a quotient, 2^-22 of itself."""
    x = delta_ref.inputs(B, H, Hk, T, d, mode, seed=T, device="cuda")
    G = torch.Generator().manual_seed(T)
    x["v"] = (x["v"].float().cpu() * size ** torch.rand(B, H, T, 1, generator=G)).to(x["v"].dtype).cuda()
    y = DeltaMemory(d, mode, B, H, k_heads=Hk).forward(x["k"], x["q"], x["v"], x["g"], x["beta"], {"W": x["W"].clone()}, attn=x["attn"])
    want, _ = delta_ref.forward(x, gated=True)
    plain, _ = delta_ref.forward(x)
    largest = plain.abs().amax((-1, -2), keepdim=True)
    bar = (2**-8 if mode == "bf16" else 2**-22) * want.abs() + delta_ref.NORM32 / 4 * x["attn"].double().abs() * largest + 1e-30
    assert ((y.double() - want).abs() / bar).max() <= 1
