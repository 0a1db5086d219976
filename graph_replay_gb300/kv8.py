"""The 8-bit K/V cache on torch tensors: e4m3 values with a power-of-two scale
for each block of positions and K/V head (graphdec.h, "The 8-bit K/V cache").

    cache = KV8Cache.empty(rows, cap, n_kv_heads, head_dim)
    cache.append(k, v, kv_len)                     # one new token for each row
    out = cache.attend(q, kv_len, window=4096, sinks=4)

Both calls launch on torch's current stream and return at once; nothing reads
back to the host.  ``check`` does, and raises if a call on any stream met an
entry of ``kv_len``, ``q_start``, the page table or the scales that is out of range.
"""
from __future__ import annotations

import threading
from typing import Optional

import torch

from . import _binding as B

_raw_stream = torch._C._cuda_getCurrentRawStream   # of a device: what torch.cuda.current_stream wraps, without the wrapper
_DT = {torch.float32: B.DEC_DTYPE_F32, torch.bfloat16: B.DEC_DTYPE_BF16}


class KV8Cache:
    """k, v: uint8 or float8_e4m3fn [num_pages, n_kv_heads, page_size, head_dim];
    k_scale, v_scale: uint8 or float8_e8m0fnu [num_pages, n_kv_heads, page_size / scale_block];
    page_table: int32 [rows, pages_per_row], or None: `rows` rows of equally many pages, in order."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                 page_table: Optional[torch.Tensor] = None, rows: int = 0):
        for t in (k, v, k_scale, v_scale) + (() if page_table is None else (page_table,)):
            if not t.is_cuda or not t.is_contiguous() or t.device != k.device:
                raise ValueError("KV8Cache: contiguous CUDA tensors on one device")
        if k.dim() != 4 or k.shape != v.shape or k.dtype not in (torch.uint8, torch.float8_e4m3fn) or v.dtype != k.dtype:
            raise ValueError("KV8Cache: k and v are e4m3 bytes [num_pages, n_kv_heads, page_size, head_dim]")
        pages, heads, page, dim = k.shape
        if (k_scale.dim() != 3 or k_scale.shape != v_scale.shape or k_scale.element_size() != 1
                or v_scale.element_size() != 1 or k_scale.shape[:2] != k.shape[:2] or k_scale.shape[2] < 1
                or page % k_scale.shape[2]):
            raise ValueError("KV8Cache: scales are bytes [num_pages, n_kv_heads, page_size / scale_block]")
        if page_table is None:
            if rows < 1 or pages % rows:
                raise ValueError("KV8Cache: without a page table, rows must divide num_pages")
            per_row = pages // rows
        else:
            if page_table.dim() != 2 or page_table.dtype != torch.int32:
                raise ValueError("KV8Cache: page_table is int32 [rows, pages_per_row]")
            rows, per_row = page_table.shape
        self.k, self.v, self.k_scale, self.v_scale, self.page_table = k, v, k_scale, v_scale, page_table
        self.rows, self.cap, self.n_kv_heads, self.head_dim = rows, per_row * page, heads, dim
        self.page_size, self.scale_block = page, page // k_scale.shape[2]
        self.device = k.device
        self._need, self._ws, self._lock = {}, {}, threading.Lock()
        self._err = torch.zeros(1, dtype=torch.int32, device=k.device)
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(k.device).synchronize()   # zeroed before a call on any other stream adds to it
        self._c = B.dec_kv8_cache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                  None if page_table is None else page_table.data_ptr(), rows, per_row, page, pages,
                                  heads, dim, self.scale_block, k.device.index)

    @classmethod
    def empty(cls, rows: int, cap: int, n_kv_heads: int, head_dim: int, scale_block: int = 64,
              device="cuda") -> "KV8Cache":
        """An empty contiguous cache of `cap` positions (a multiple of scale_block) for each row."""
        if scale_block < 1 or cap < 1 or cap % scale_block:
            raise ValueError(f"KV8Cache.empty: cap {cap} is no multiple of scale_block {scale_block}")
        k = torch.zeros(rows, n_kv_heads, cap, head_dim, dtype=torch.uint8, device=device)
        s = torch.full((rows, n_kv_heads, cap // scale_block), 127, dtype=torch.uint8, device=device)
        return cls(k, torch.zeros_like(k), s, s.clone(), rows=rows)

    def _batch(self, kv_len, q_start, total, max_new):
        for t in (kv_len,) if q_start is None else (kv_len, q_start):
            if t.dtype != torch.int32 or t.device != self.device or not t.is_contiguous():
                raise ValueError("KV8Cache: kv_len and q_start are contiguous int32 tensors on the cache's device")
        if not -0x80000000 <= max_new <= 0x7FFFFFFF:
            B.check_int32(max_new=max_new)
        if kv_len.numel() != self.rows or (q_start is not None and q_start.numel() != self.rows + 1):
            raise ValueError("KV8Cache: kv_len has rows entries, q_start rows + 1")
        return B.dec_kv8_batch(None if q_start is None else q_start.data_ptr(), kv_len.data_ptr(),
                               self._err.data_ptr(), total, max_new)

    def _tokens(self, what, t, heads):
        shape, stride = t.shape, t.stride()
        if (len(shape) != 3 or t.dtype not in _DT or t.device != self.device or shape[2] != self.head_dim
                or (heads and shape[1] != heads) or stride[2] != 1 or stride[1] != self.head_dim):
            raise ValueError(f"KV8Cache: {what} is f32 or bf16 [tokens, heads, head_dim], heads side by side, on the "
                             "cache's device")
        return stride[0] if shape[0] > 1 else shape[1] * shape[2]

    def append(self, k: torch.Tensor, v: torch.Tensor, kv_len: torch.Tensor, q_start: Optional[torch.Tensor] = None,
               max_new: int = 1) -> None:
        """Store new K and V [tokens, n_kv_heads, head_dim].  kv_len [rows] counts each row's positions, these
        tokens included; q_start [rows + 1] gives each row its packed tokens (None: one each), at most max_new."""
        if k.shape != v.shape or k.dtype != v.dtype:
            raise ValueError("KV8Cache: k and v have one shape and type")
        ks, vs = self._tokens("k", k, self.n_kv_heads), self._tokens("v", v, self.n_kv_heads)
        b = self._batch(kv_len, q_start, k.shape[0], max_new)
        n = B.dec_kv8_new(k.data_ptr(), v.data_ptr(), ks, vs, _DT[k.dtype], 0)
        B.dec_kv8_append(self._c, b, n, _raw_stream(self._c.device))

    def workspace_bytes(self, tokens: int, n_heads: int, max_new: int = 1, window: int = 0, sinks: int = 0,
                        dtype: torch.dtype = torch.bfloat16) -> int:
        """Bytes of workspace that attend needs for these sizes."""
        key = (tokens, n_heads, max_new, window, sinks, dtype)
        need = self._need.get(key)
        if need is None:
            B.check_int32(tokens=tokens, n_heads=n_heads, max_new=max_new, window=window, sinks=sinks)
            b = B.dec_kv8_batch(self._c.pages or self._c.k, self._c.k, self._c.k, tokens, max_new)   # addresses are not read
            a = B.dec_kv8_attn(self._c.k, self._c.k, n_heads * self.head_dim, n_heads * self.head_dim, _DT[dtype], n_heads,
                               window, sinks, 0.0, None, 0)
            if len(self._need) >= 256:   # prompts come in any length
                self._need.clear()
            need = self._need[key] = B.dec_kv8_workspace(self._c, b, a)
        return need

    def _workspace(self, stream: int, need: int) -> torch.Tensor:
        # One for each stream, zeroed once: calls on a stream follow one another, and each leaves it as it found it.  A
        # recorded graph gets its own, from its pool, and zeroes the counters when it runs
        if torch.cuda.is_current_stream_capturing():
            ws = torch.empty(need, dtype=torch.uint8, device=self.device)
            ws[:-(-self.rows * self.n_kv_heads * 4 // 256) * 256].zero_()
            return ws
        ws = self._ws.get(stream)
        if ws is None or ws.numel() < need:
            ws = self._ws[stream] = torch.zeros(need, dtype=torch.uint8, device=self.device)
        return ws

    def attend(self, q: torch.Tensor, kv_len: torch.Tensor, q_start: Optional[torch.Tensor] = None, max_new: int = 1,
               window: int = 0, sinks: int = 0, scale: float = 0.0, out: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Attention of q [tokens, n_heads, head_dim] over the cache, causal; with a window each token sees its last
        `window` positions (its own among them) and the first `sinks`.  scale 0: 1 / sqrt(head_dim).  Returns `out`
        (allocated like q if None); packed tokens that belong to no row are not written.  `workspace`: uint8, zeroed
        before its first use, of workspace_bytes(...); None: the cache keeps one for each stream, and a graph that
        records the call one of its own."""
        if not (-0x80000000 <= window <= 0x7FFFFFFF and -0x80000000 <= sinks <= 0x7FFFFFFF):
            B.check_int32(window=window, sinks=sinks)
        qs = self._tokens("q", q, 0)
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        elif out.shape != q.shape or out.dtype != q.dtype:
            raise ValueError("KV8Cache: out has q's shape and type")
        os_ = self._tokens("out", out, 0)
        tokens, heads, _ = q.shape
        b = self._batch(kv_len, q_start, tokens, max_new)
        stream = _raw_stream(self._c.device)
        if workspace is not None and (workspace.device != self.device or not workspace.is_contiguous()):
            raise ValueError("KV8Cache: the workspace is contiguous and on the cache's device")
        with self._lock:   # a call may launch two kernels that hand on the workspace: another thread's come before or after
            if workspace is None:
                workspace = self._workspace(stream, self.workspace_bytes(tokens, heads, max_new, window, sinks, q.dtype))
            a = B.dec_kv8_attn(q.data_ptr(), out.data_ptr(), qs, os_, _DT[q.dtype], heads, window, sinks, scale,
                               workspace.data_ptr(), workspace.numel() * workspace.element_size())
            B.dec_kv8_attend(self._c, b, a, stream)
        return out

    def check(self) -> None:
        """Wait for all work on the device so far, on whatever stream and in whatever graph, and raise DecError if a call
        met an entry out of range since the last check.  Not while any stream is being captured."""
        torch.cuda.synchronize(self.device)
        bits = int(self._err.item())
        if bits:
            self._err.zero_()
            torch.cuda.synchronize(self.device)   # a later call on another stream adds its bits after this
            raise B.DecError(B.DEC_E_DEVICE_FAULT, f"8-bit K/V cache: an entry out of range (error word 0x{bits:x})")
