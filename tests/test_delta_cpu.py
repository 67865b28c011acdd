"""Refusals of the gated delta rule's and the paged cache's calls: all before anything touches a GPU."""
import ctypes

import pytest
import torch

import delta_ref
from titans_long_term_b200 import DeltaMemory, TitansError, mem

GOOD = dict(d=64, mode=mem.BF16, B=2, H=4, Hk=2)


def config(**other):
    c = {**GOOD, **other}
    return mem.DeltaConfig(c["d"], c["mode"], c["B"], c["H"], c["Hk"])


@pytest.mark.parametrize("other,status", [
    (dict(d=96), mem.EUNSUPPORTED), (dict(mode=3), mem.EINVAL), (dict(B=0), mem.EINVAL), (dict(H=-1), mem.EINVAL),
    (dict(Hk=0), mem.EINVAL), (dict(Hk=3), mem.EINVAL), (dict(B=1 << 20, H=32), mem.EINVAL)])
def test_bad_configurations(other, status):
    L, c = mem.lib(), config(**other)
    p = [16] * 6
    assert L.titans_delta_forward(ctypes.byref(c), *p, 4, *[16] * 4, 1 << 40, None) == status
    assert L.titans_delta_step(ctypes.byref(c), *[16] * 8, None) == status
    assert L.titans_delta_backward(ctypes.byref(c), *p, 4, *[16] * 10, 1 << 40, None) == status
    assert L.titans_delta_workspace_bytes(ctypes.byref(c), 4, 0) == ctypes.c_size_t(-1).value
    assert L.titans_last_error_string().decode()


def test_null_configuration():
    L = mem.lib()
    assert L.titans_delta_forward(None, *[16] * 6, 4, *[16] * 4, 0, None) == mem.EINVAL
    assert L.titans_delta_workspace_bytes(None, 4, 0) == ctypes.c_size_t(-1).value


@pytest.mark.parametrize("T,status", [(0, mem.EINVAL), (-5, mem.EINVAL), (1 << 25, mem.EUNSUPPORTED)])
def test_bad_lengths(T, status):
    L, c = mem.lib(), config()
    assert L.titans_delta_forward(ctypes.byref(c), *[16] * 6, T, *[16] * 4, 1 << 40, None) == status
    assert L.titans_delta_backward(ctypes.byref(c), *[16] * 6, T, *[16] * 10, 1 << 40, None) == status
    assert L.titans_delta_workspace_bytes(ctypes.byref(c), T, 0) == ctypes.c_size_t(-1).value
    assert L.titans_delta_workspace_bytes(ctypes.byref(c), 4, 2) == ctypes.c_size_t(-1).value


@pytest.mark.parametrize("bad", [None, 8, 2])
@pytest.mark.parametrize("at", [0, 1, 2, 7, 9])  # k, q, v, W, y
def test_forward_pointers(at, bad):
    L, c = mem.lib(), config()
    args = [16] * 6 + [300] + [16] * 4
    args[at] = bad
    assert L.titans_delta_forward(ctypes.byref(c), *args, 1 << 40, None) == mem.EINVAL


@pytest.mark.parametrize("at", [3, 4])  # g, beta
def test_gate_pointers(at):
    L, c = mem.lib(), config()
    for bad in (None, 2):
        args = [16] * 6 + [300] + [16] * 4
        args[at] = bad
        assert L.titans_delta_forward(ctypes.byref(c), *args, 1 << 40, None) == mem.EINVAL
        args = [16] * 8
        args[at] = bad
        assert L.titans_delta_step(ctypes.byref(c), *args, None) == mem.EINVAL


def test_backward_pointers():
    L, c = mem.lib(), config()
    for at in (0, 1, 2, 3, 4, 7, 8, 10, 11, 12, 13, 14, 15, 16):
        args = [16] * 6 + [300] + [16] * 10
        args[at] = None
        assert L.titans_delta_backward(ctypes.byref(c), *args, 1 << 40, None) == mem.EINVAL, at


def test_small_workspaces():
    L, c = mem.lib(), config()
    for call, f, n in ((0, L.titans_delta_forward, 4), (1, L.titans_delta_backward, 10)):
        need = L.titans_delta_workspace_bytes(ctypes.byref(c), 1000, call)
        if need:
            assert f(ctypes.byref(c), *[16] * 6, 1000, *[16] * n, need - 1, None) == mem.EINVAL
            assert "workspace" in L.titans_last_error_string().decode()


def test_binding_refuses():
    with pytest.raises(TitansError):
        DeltaMemory(96, "bf16", 1, 4)
    with pytest.raises(TitansError):
        DeltaMemory(64, "bf16", 1, 4, k_heads=3)
    with pytest.raises(ValueError):
        DeltaMemory(64, "fp16", 1, 4)
    m = DeltaMemory(64, "bf16", 1, 4)
    with pytest.raises(TitansError) as e:
        m._workspace_bytes(1 << 25, 0)
    assert e.value.status == mem.EUNSUPPORTED and "2^31" in str(e.value)
    x = delta_ref.inputs(1, 4, 4, 8, 64, "bf16")
    with pytest.raises(ValueError, match="CUDA"):
        m.forward(x["k"], x["q"], x["v"], x["g"], x["beta"], {"W": x["W"]})


def test_reference_gradients_against_differences():
    """The 64-bit adjoint the GPU tests compare with, against central differences of the 64-bit forward."""
    x = delta_ref.inputs(2, 4, 2, 9, 4, "fp32", seed=3)
    x["lengths"] = torch.tensor([9, 6], dtype=torch.int32)
    x = {n: t.double() if t.is_floating_point() else t for n, t in x.items()}

    def value(z):
        y, W = delta_ref.forward(z)
        return float((y * x["dy"]).sum() + (W * x["dW"]).sum())

    out = delta_ref.backward(x)
    G = torch.Generator().manual_seed(7)
    for n in ("k", "q", "v", "g", "beta", "W"):
        way = torch.randn(x[n].shape, generator=G, dtype=torch.float64)
        h = 1e-5
        change = (value({**x, n: x[n] + h * way}) - value({**x, n: x[n] - h * way})) / (2 * h)
        assert abs(change - float((out[n] * way).sum())) <= 1e-7 * max(1.0, abs(change)), n
