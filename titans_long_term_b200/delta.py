"""Gated delta rule: Python binding of the titans_delta_* calls of include/titans_mem.h."""
from __future__ import annotations

import ctypes
from typing import Dict, Optional

import torch

from .mem import BF16, FP32, DeltaConfig, TitansError, _check, lib


def _need(name: str, t: torch.Tensor, dtype: torch.dtype, shape: tuple, device: torch.device):
    if t.dtype != dtype or t.device != device or not t.is_contiguous() or t.shape != shape:
        raise ValueError(f"{name}: expected contiguous {dtype} of shape {shape} on {device}")


def _device(t: torch.Tensor) -> torch.device:
    if not t.is_cuda:
        raise ValueError("expected CUDA tensors")
    return t.device


class _On:
    """Makes `stream` (None: the current one) of the tensors' device current, so that what the call allocates
    belongs to it, and gives its handle."""

    __slots__ = ("guard", "handle")

    def __init__(self, device: torch.device, stream: Optional[torch.cuda.Stream]):
        if stream is not None:
            if stream.device != device:
                raise ValueError(f"the stream is on {stream.device}, the tensors are on {device}")
            self.guard = torch.cuda.stream(stream)
            self.handle = stream.cuda_stream
        else:
            self.guard = None if torch.cuda.current_device() == device.index else torch.cuda.device(device)
            self.handle = torch.cuda.current_stream(device).cuda_stream

    def __enter__(self) -> int:
        if self.guard is not None:
            self.guard.__enter__()
        return self.handle

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


class DeltaMemory:
    """B*H units of a gated-delta-rule memory: per token A = exp(g) W, e = beta (v - A k), W = A + e k^T,
    y = W q. `mode` ("bf16" or "fp32") is the dtype of k, q, v, attn and y; W, g and beta are fp32.
    `k_heads` key/query heads (default H) are shared by H / k_heads value heads each. Tensors are contiguous
    and on one CUDA device, whichever is current. Calls keep nothing between them."""

    def __init__(self, d: int, mode: str, B: int, H: int, k_heads: Optional[int] = None):
        if mode not in ("bf16", "fp32"):
            raise ValueError(f"mode: expected 'bf16' or 'fp32', got {mode!r}")
        self.d, self.mode, self.B, self.H = d, mode, B, H
        self.k_heads = H if k_heads is None else k_heads
        self.dtype = torch.bfloat16 if mode == "bf16" else torch.float32
        self._cfg = DeltaConfig(d, BF16 if mode == "bf16" else FP32, B, H, self.k_heads)
        self._ref = ctypes.byref(self._cfg)
        self._bytes: Dict[tuple, int] = {}
        self._workspace_bytes(1, 0)  # refuses a bad configuration here

    def _workspace_bytes(self, T: int, call: int) -> int:
        n = self._bytes.get((T, call))
        if n is None:
            n = lib().titans_delta_workspace_bytes(self._ref, T, call)
            if n == ctypes.c_size_t(-1).value:
                msg = lib().titans_last_error_string().decode()
                raise TitansError(lib().titans_delta_step(self._ref, *[None] * 8, None), msg)
            self._bytes[(T, call)] = n
        return n

    def new_state(self, device="cuda") -> Dict[str, torch.Tensor]:
        """An empty memory: {"W": zeros [B, H, d, d]}."""
        return {"W": torch.zeros(self.B, self.H, self.d, self.d, device=device)}

    def _inputs(self, k, q, v, g, beta, W, T, lengths):
        B, H, Hk, d = self.B, self.H, self.k_heads, self.d
        dev = _device(k)
        t = () if T is None else (T,)
        _need("k", k, self.dtype, (B, Hk, *t, d), dev)
        _need("q", q, self.dtype, (B, Hk, *t, d), dev)
        _need("v", v, self.dtype, (B, H, *t, d), dev)
        _need("g", g, torch.float32, (B, H, *t), dev)
        _need("beta", beta, torch.float32, (B, H, *t), dev)
        _need("W", W, torch.float32, (B, H, d, d), dev)
        if lengths is not None:
            _need("lengths", lengths, torch.int32, (B,), dev)
        return dev

    def forward(self, k, q, v, g, beta, state: Dict[str, torch.Tensor], lengths: Optional[torch.Tensor] = None,
                attn: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """k, q [B, k_heads, T, d]; v [B, H, T, d]; g (log of what is retained, <= 0) and beta [B, H, T];
        state {"W": [B, H, d, d]} updated in place; `lengths` [B] int32: the tokens that count, the others
        have y = 0. Returns y [B, H, T, d], or attn * sigmoid(y) with `attn`."""
        W, T = state["W"], v.shape[-2]
        dev = self._inputs(k, q, v, g, beta, W, T, lengths)
        if attn is not None:
            _need("attn", attn, self.dtype, v.shape, dev)
        with _On(dev, stream) as st:
            if y is None:
                y = torch.empty_like(v)
            else:
                _need("y", y, self.dtype, v.shape, dev)
            n = self._workspace_bytes(T, 0)
            ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
            _check(lib().titans_delta_forward(
                self._ref, k.data_ptr(), q.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
                None if lengths is None else lengths.data_ptr(), T, W.data_ptr(),
                None if attn is None else attn.data_ptr(), y.data_ptr(), None if ws is None else ws.data_ptr(), n, st))
        return y

    def step(self, k, q, v, g, beta, state: Dict[str, torch.Tensor], attn: Optional[torch.Tensor] = None,
             y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """One token: k, q [B, k_heads, d]; v, attn [B, H, d]; g, beta [B, H]; state updated in place;
        returns y [B, H, d]."""
        W = state["W"]
        dev = self._inputs(k, q, v, g, beta, W, None, None)
        if attn is not None:
            _need("attn", attn, self.dtype, v.shape, dev)
        with _On(dev, stream) as st:
            if y is None:
                y = torch.empty_like(v)
            else:
                _need("y", y, self.dtype, v.shape, dev)
            _check(lib().titans_delta_step(self._ref, k.data_ptr(), q.data_ptr(), v.data_ptr(), g.data_ptr(),
                                           beta.data_ptr(), W.data_ptr(), None if attn is None else attn.data_ptr(),
                                           y.data_ptr(), st))
        return y

    def backward(self, k, q, v, g, beta, state: Dict[str, torch.Tensor], dy: torch.Tensor,
                 dstate: Optional[Dict[str, torch.Tensor]] = None, lengths: Optional[torch.Tensor] = None,
                 stream=None) -> Dict[str, torch.Tensor]:
        """Gradients of <dy, y> + <dstate["W"], final W> for forward() without attn from `state` (read only).
        Returns a dict with keys k, q, v, g, beta and W; those of shared key heads are summed."""
        W, T = state["W"], v.shape[-2]
        dev = self._inputs(k, q, v, g, beta, W, T, lengths)
        _need("dy", dy, self.dtype, v.shape, dev)
        dW = None if dstate is None else dstate.get("W")
        if dW is not None:
            _need("dstate W", dW, torch.float32, W.shape, dev)
        with _On(dev, stream) as st:
            out = {"k": torch.empty_like(k), "q": torch.empty_like(q), "v": torch.empty_like(v),
                   "g": torch.empty_like(g), "beta": torch.empty_like(beta), "W": torch.empty_like(W)}
            n = self._workspace_bytes(T, 1)
            ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
            _check(lib().titans_delta_backward(
                self._ref, k.data_ptr(), q.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
                None if lengths is None else lengths.data_ptr(), T, W.data_ptr(), dy.data_ptr(),
                None if dW is None else dW.data_ptr(), out["k"].data_ptr(), out["q"].data_ptr(), out["v"].data_ptr(),
                out["g"].data_ptr(), out["beta"].data_ptr(), out["W"].data_ptr(),
                None if ws is None else ws.data_ptr(), n, st))
        return out
