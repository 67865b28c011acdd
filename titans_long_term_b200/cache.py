"""Paged key/value cache and its attention: Python binding of the titans_cache_* calls of include/titans_mem.h."""
from __future__ import annotations

import ctypes
import math
from typing import Dict, Optional, Tuple

import torch

from .delta import _F32, _I32, _need, _On, _run
from .mem import CacheConfig, CachePages, _check, lib

TYPES = {"bf16": (0, torch.bfloat16), "e4m3": (1, torch.float8_e4m3fn)}


class PagedCache:
    """Keys and values of B sequences in pages, and the attention of new tokens over them. Token p of sequence b
    lies in page table[b, p // page], slot p % page. `dtype` "bf16", or "e4m3": 8 bits with one power-of-two
    scale per token and head, set as the token is written. H query heads share `kv_heads` key/value heads
    (default H). The tensors are the caller's; the handle belongs to the device that is current here, and is kept as
    long as graphs that its calls were captured into are replayed."""

    def __init__(self, d: int, dtype: str, B: int, H: int, kv_heads: Optional[int] = None, page: int = 64,
                 num_pages: int = 0, max_pages: int = 0):
        if dtype not in TYPES:
            raise ValueError(f"dtype: expected 'bf16' or 'e4m3', got {dtype!r}")
        self.d, self.B, self.H, self.page = d, B, H, page
        self.kv_heads = H if kv_heads is None else kv_heads
        self.num_pages, self.max_pages = num_pages, max_pages
        kind, self.dtype = TYPES[dtype]
        self.scaled = dtype == "e4m3"
        self._cfg = CacheConfig(d, kind, B, H, self.kv_heads, page, num_pages, max_pages)
        self._bytes: Dict[int, int] = {}
        h = ctypes.c_void_p()
        _check(lib().titans_cache_init(ctypes.byref(self._cfg), ctypes.byref(h)))
        self._h = h
        self._lib = lib()
        self._index = torch.cuda.current_device()
        self.device = torch.device("cuda", self._index)
        self._pool, self._table, self._batch = (num_pages, self.kv_heads, page, d), (B, max_pages), (B,)

    def close(self):
        if getattr(self, "_h", None):
            lib().titans_cache_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def new_pages(self) -> Dict[str, torch.Tensor]:
        """An empty pool: k, v [num_pages, kv_heads, page, d] and, for e4m3, k_scale, v_scale [.., page] fp32."""
        shape = (self.num_pages, self.kv_heads, self.page, self.d)
        p = {n: torch.zeros(shape, dtype=torch.uint8 if self.scaled else self.dtype, device=self.device)
             for n in ("k", "v")}
        if self.scaled:
            p = {n: t.view(self.dtype) for n, t in p.items()}
            p |= {n: torch.ones(shape[:-1], device=self.device) for n in ("k_scale", "v_scale")}
        return p

    def _where(self, pages, table, starts, counts) -> CachePages:
        k, v = pages["k"], pages["v"]
        _need(self._index, ("pages k", k, self.dtype, self._pool), ("pages v", v, self.dtype, self._pool),
              ("table", table, _I32, self._table), ("starts", starts, _I32, self._batch))
        if counts is not None:
            _need(self._index, ("counts", counts, _I32, self._batch))
        if not self.scaled:
            return CachePages(k.data_ptr(), v.data_ptr())
        ks, vs = pages["k_scale"], pages["v_scale"]
        _need(self._index, ("pages k_scale", ks, _F32, self._pool[:-1]), ("pages v_scale", vs, _F32, self._pool[:-1]))
        return CachePages(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr())

    def append(self, k, v, pages: Dict[str, torch.Tensor], table, starts, counts: Optional[torch.Tensor] = None,
               stream=None) -> None:
        """Writes k, v [B, kv_heads, T, d] bf16 at positions starts[b] + t, t < counts[b] (None: all T)."""
        T, shape = k.shape[-2], (self.B, self.kv_heads, k.shape[-2], self.d)
        _need(self._index, ("k", k, torch.bfloat16, shape), ("v", v, torch.bfloat16, shape))
        p = self._where(pages, table, starts, counts)
        _run(self._index, stream, lambda st: _check(self._lib.titans_cache_append(
            self._h, k.data_ptr(), v.data_ptr(), T, ctypes.byref(p), table.data_ptr(), starts.data_ptr(),
            None if counts is None else counts.data_ptr(), st)))

    def read(self, pages: Dict[str, torch.Tensor], table, starts, T: int, counts: Optional[torch.Tensor] = None,
             stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
        """k, v [B, kv_heads, T, d] bf16 of positions starts[b] + t; zeros for t >= counts[b]."""
        if T < 1:
            raise ValueError(f"T: expected at least 1, got {T}")
        p = self._where(pages, table, starts, counts)

        def call(st):
            both = torch.empty(2, self.B, self.kv_heads, T, self.d, dtype=torch.bfloat16, device=self.device)
            k, v = both.unbind()
            _check(self._lib.titans_cache_read(self._h, ctypes.byref(p), table.data_ptr(), starts.data_ptr(),
                                               None if counts is None else counts.data_ptr(), T, k.data_ptr(),
                                               v.data_ptr(), st))
            return k, v

        return _run(self._index, stream, call)

    def attend(self, q, pages: Dict[str, torch.Tensor], table, starts, counts: Optional[torch.Tensor] = None,
               window: int = 0, sinks: int = 0, scale: Optional[float] = None, o: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
        """Attention of q [B, H, T, d] at positions p = starts[b] + t over the cached keys j <= p, with
        `window` > 0 only those with j > p - window or j < sinks; scale defaults to d^-1/2. Rows t >= counts[b]
        are zeros. Returns o [B, H, T, d] bf16, ready to be the `attn` of a gated memory."""
        T, shape = q.shape[-2], (self.B, self.H, q.shape[-2], self.d)
        if max(abs(window), abs(sinks)) >= 1 << 31:  # beyond any position, and what the call's int holds
            raise ValueError(f"window and sinks: expected magnitudes below 2^31, got {window} and {sinks}")
        _need(self._index, ("q", q, torch.bfloat16, shape))
        if o is not None:
            _need(self._index, ("o", o, torch.bfloat16, shape))
        p = self._where(pages, table, starts, counts)
        n = self._bytes.get(T)
        if n is None:
            n = self._bytes[T] = self._lib.titans_cache_attend_workspace_bytes(self._h, T)

        def call(st):
            out = torch.empty_like(q) if o is None else o
            ws = torch.empty(n, dtype=torch.uint8, device=self.device) if n else None
            _check(self._lib.titans_cache_attend(
                self._h, q.data_ptr(), T, ctypes.byref(p), table.data_ptr(), starts.data_ptr(),
                None if counts is None else counts.data_ptr(), window, sinks,
                1.0 / math.sqrt(self.d) if scale is None else scale, out.data_ptr(),
                None if ws is None else ws.data_ptr(), n, st))
            return out

        return _run(self._index, stream, call)

    def sync_status(self, stream=None):
        """Waits for the stream; raises TitansError if a call met a missing page since the last one."""
        with _On(self._index, stream) as st:
            _check(self._lib.titans_cache_sync_status(self._h, st))
