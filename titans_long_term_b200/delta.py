"""Gated delta rule: Python binding of the titans_delta_* calls of include/titans_mem.h."""
from __future__ import annotations

import ctypes
from typing import Dict, Optional

import torch

from .mem import BF16, FP32, DeltaConfig, TitansError, _check, lib


_raw_stream = torch._C._cuda_getCurrentRawStream  # handle of a device's current stream
_F32, _I32 = torch.float32, torch.int32


def _need(index: int, *wanted) -> None:
    """Each (name, tensor, dtype, shape) has to be contiguous and on CUDA device `index`."""
    for name, t, dtype, shape in wanted:
        if t.dtype is not dtype or t.shape != shape or t.get_device() != index or index < 0 or not t.is_contiguous():
            raise ValueError(f"{name}: expected contiguous {dtype} of shape {tuple(shape)} on CUDA device {index}, "
                             f"got {t.dtype} of shape {tuple(t.shape)} on {t.device}" if index >= 0 else
                             "expected CUDA tensors")


class _On:
    """Makes `stream` (None: the current one) of device `index` current, so that what a call allocates belongs to it,
    and gives its handle."""

    __slots__ = ("guard", "handle")

    def __init__(self, index: int, stream: Optional[torch.cuda.Stream]):
        if stream is not None:
            if stream.device_index != index:
                raise ValueError(f"the stream is on device {stream.device_index}, the tensors are on device {index}")
            self.guard = torch.cuda.stream(stream)
            self.handle = stream.cuda_stream
        else:
            self.guard = torch.cuda.device(index)
            self.handle = _raw_stream(index)

    def __enter__(self) -> int:
        self.guard.__enter__()
        return self.handle

    def __exit__(self, *exc):
        self.guard.__exit__(*exc)


def _run(index: int, stream: Optional[torch.cuda.Stream], call):
    """call(stream handle) with device `index` and `stream` current; nothing to change is the common case."""
    if stream is None and torch._C._cuda_getDevice() == index:
        return call(_raw_stream(index))
    with _On(index, stream) as handle:
        return call(handle)


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
        self._lib = lib()
        self._step_shapes = ((B, self.k_heads, d), (B, H, d), (B, H), (B, H, d, d))
        self._workspace_bytes(1, 0)  # refuses a bad configuration here

    def _workspace_bytes(self, T: int, call: int) -> int:
        n = self._bytes.get((T, call))
        if n is None:
            n = lib().titans_delta_workspace_bytes(self._ref, T, call)
            if n == ctypes.c_size_t(-1).value:
                msg = lib().titans_last_error_string().decode()
                # the call itself refuses the configuration and T before anything else, with the status for it
                raise TitansError(lib().titans_delta_forward(self._ref, *[None] * 6, T, *[None] * 4, 0, None), msg)
            self._bytes[(T, call)] = n
        return n

    def new_state(self, device="cuda") -> Dict[str, torch.Tensor]:
        """An empty memory: {"W": zeros [B, H, d, d]}."""
        return {"W": torch.zeros(self.B, self.H, self.d, self.d, device=device)}

    def forward(self, k, q, v, g, beta, state: Dict[str, torch.Tensor], lengths: Optional[torch.Tensor] = None,
                attn: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """k, q [B, k_heads, T, d]; v [B, H, T, d]; g (log of what is retained, <= 0) and beta [B, H, T];
        state {"W": [B, H, d, d]} updated in place; `lengths` [B] int32: the tokens that count, the others
        have y = 0. Returns y [B, H, T, d], or attn * sigmoid(y) with `attn`."""
        W, T, index = state["W"], v.shape[-2], v.get_device()
        B, H, d, tok = self.B, self.H, self.d, self.dtype
        keys, values, gates = (B, self.k_heads, T, d), (B, H, T, d), (B, H, T)
        _need(index, ("k", k, tok, keys), ("q", q, tok, keys), ("v", v, tok, values), ("g", g, _F32, gates),
              ("beta", beta, _F32, gates), ("W", W, _F32, (B, H, d, d)))
        if lengths is not None:
            _need(index, ("lengths", lengths, _I32, (B,)))
        if attn is not None:
            _need(index, ("attn", attn, tok, values))
        if y is not None:
            _need(index, ("y", y, tok, values))
        n = self._workspace_bytes(T, 0)

        def call(st):
            out = torch.empty_like(v) if y is None else y
            ws = torch.empty(n, dtype=torch.uint8, device=v.device) if n else None
            _check(lib().titans_delta_forward(
                self._ref, k.data_ptr(), q.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
                None if lengths is None else lengths.data_ptr(), T, W.data_ptr(),
                None if attn is None else attn.data_ptr(), out.data_ptr(), None if ws is None else ws.data_ptr(), n, st))
            return out

        return _run(index, stream, call)

    def step(self, k, q, v, g, beta, state: Dict[str, torch.Tensor], attn: Optional[torch.Tensor] = None,
             y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """One token: k, q [B, k_heads, d]; v, attn [B, H, d]; g, beta [B, H]; state updated in place;
        returns y [B, H, d]."""
        W, index, tok = state["W"], v.get_device(), self.dtype
        keys, values, gates, matrix = self._step_shapes
        _need(index, ("k", k, tok, keys), ("q", q, tok, keys), ("v", v, tok, values), ("g", g, _F32, gates),
              ("beta", beta, _F32, gates), ("W", W, _F32, matrix))
        if attn is not None:
            _need(index, ("attn", attn, tok, values))
        if y is not None:
            _need(index, ("y", y, tok, values))

        def call(st):
            out = torch.empty_like(v) if y is None else y
            status = self._lib.titans_delta_step(self._ref, k.data_ptr(), q.data_ptr(), v.data_ptr(), g.data_ptr(),
                                                 beta.data_ptr(), W.data_ptr(),
                                                 None if attn is None else attn.data_ptr(), out.data_ptr(), st)
            if status:
                _check(status)
            return out

        return _run(index, stream, call)

    def backward(self, k, q, v, g, beta, state: Dict[str, torch.Tensor], dy: torch.Tensor,
                 dstate: Optional[Dict[str, torch.Tensor]] = None, lengths: Optional[torch.Tensor] = None,
                 stream=None) -> Dict[str, torch.Tensor]:
        """Gradients of <dy, y> + <dstate["W"], final W> for forward() without attn from `state` (read only).
        Returns a dict with keys k, q, v, g, beta and W; those of shared key heads are summed."""
        W, T, index = state["W"], v.shape[-2], v.get_device()
        B, H, d, tok = self.B, self.H, self.d, self.dtype
        keys, values, gates, matrix = (B, self.k_heads, T, d), (B, H, T, d), (B, H, T), (B, H, d, d)
        _need(index, ("k", k, tok, keys), ("q", q, tok, keys), ("v", v, tok, values), ("g", g, _F32, gates),
              ("beta", beta, _F32, gates), ("W", W, _F32, matrix), ("dy", dy, tok, values))
        dW = None if dstate is None else dstate.get("W")
        if dW is not None:
            _need(index, ("dstate W", dW, _F32, matrix))
        if lengths is not None:
            _need(index, ("lengths", lengths, _I32, (B,)))
        n = self._workspace_bytes(T, 1)

        def call(st):
            out = {"k": torch.empty_like(k), "q": torch.empty_like(q), "v": torch.empty_like(v),
                   "g": torch.empty_like(g), "beta": torch.empty_like(beta), "W": torch.empty_like(W)}
            ws = torch.empty(n, dtype=torch.uint8, device=v.device)
            _check(lib().titans_delta_backward(
                self._ref, k.data_ptr(), q.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
                None if lengths is None else lengths.data_ptr(), T, W.data_ptr(), dy.data_ptr(),
                None if dW is None else dW.data_ptr(), out["k"].data_ptr(), out["q"].data_ptr(), out["v"].data_ptr(),
                out["g"].data_ptr(), out["beta"].data_ptr(), out["W"].data_ptr(), ws.data_ptr(), n, st))
            return out

        return _run(index, stream, call)
