"""Matrices in 4 bits on torch tensors: codes -8 .. 7 with a bf16 scale for each group of columns of a row
(graphdec.h, "4-bit weights").

    w = W4Weight.quantize(weight, group=128)              # weight [n, k]
    y = w.linear(x, norm=gain, residual=h)                # h + W rmsnorm(x), one launch for a few tokens
    a = gate.glu(up, x, act="silu", norm=gain)            # silu(gate x) * (up x)

The calls launch on torch's current stream and return at once; nothing reads back to the host.  ``check`` does, and
raises if a call on any stream gave up waiting for a copy or a product.  There is no backward pass: where gradients are
recorded, tensors that require one are refused.
"""
from __future__ import annotations

import threading
from typing import Optional

import torch

from . import _binding as B

_raw_stream = torch._C._cuda_getCurrentRawStream   # of a device: what torch.cuda.current_stream wraps, without the wrapper
_capturing = torch.cuda.is_current_stream_capturing
_DT = {torch.float32: B.DEC_DTYPE_F32, torch.bfloat16: B.DEC_DTYPE_BF16}
_ACT = {"silu": B.DEC_ACT_SILU, "gelu_tanh": B.DEC_ACT_GELU_TANH}


class _Device:
    """What the calls on one device share: the error word."""

    _all, _guard = {}, threading.Lock()

    def __init__(self, index: int):
        if _capturing():
            raise RuntimeError("W4Weight: the first one on a device is made before a stream is captured")
        self.index = index
        self.err = torch.zeros(1, dtype=torch.int32, device=f"cuda:{index}")
        self.err_ptr = self.err.data_ptr()
        torch.cuda.current_stream(self.err.device).synchronize()   # zeroed before a call on any other stream adds to it

    @classmethod
    def of(cls, index: int) -> "_Device":
        with cls._guard:
            d = cls._all.get(index)
            if d is None:
                d = cls._all[index] = cls(index)
            return d


class W4Weight:
    """codes: uint8 [n, k / 2]; scales: bfloat16 [n, k / group], group 32, 64 or 128."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor):
        for t in (codes, scales):
            if not t.is_cuda or not t.is_contiguous() or t.device != codes.device or t.dim() != 2:
                raise ValueError("W4Weight: contiguous CUDA matrices on one device")
        if codes.dtype != torch.uint8 or scales.dtype != torch.bfloat16 or codes.shape[0] != scales.shape[0]:
            raise ValueError("W4Weight: codes are uint8 [n, k / 2], scales bfloat16 [n, k / group]")
        n, k = codes.shape[0], 2 * codes.shape[1]
        if scales.shape[1] < 1 or k % scales.shape[1] or k // scales.shape[1] not in (32, 64, 128):
            raise ValueError(f"W4Weight: {scales.shape[1]} scales for {k} columns: groups are of 32, 64 or 128")
        self.codes, self.scales = codes, scales
        self.shape, self.group, self.device = (n, k), k // scales.shape[1], codes.device
        self._dev = _Device.of(codes.device.index)
        self._calls, self._lock = {}, threading.Lock()
        self._c = B.dec_w4_weight(codes.data_ptr(), scales.data_ptr(), n, k, self.group, codes.device.index)

    @classmethod
    def quantize(cls, w: torch.Tensor, group: int = 128, codes: Optional[torch.Tensor] = None,
                 scales: Optional[torch.Tensor] = None) -> "W4Weight":
        """w [n, k] (f32 or bf16; its rows may be parts of longer ones, and start at multiples of 16 bytes) in 4 bits: over each
        group scale = bf16(max |w| / 7), code = w / scale to the nearest whole number.  Into `codes` and `scales`, or new
        tensors; neither lies over w."""
        if w.dim() != 2 or not w.is_cuda or w.dtype not in _DT or w.stride(1) != 1:
            raise ValueError("W4Weight.quantize: w is an f32 or bf16 CUDA matrix, its columns side by side")
        n, k = w.shape
        if group not in (32, 64, 128) or k < 1 or k % group or n < 1:
            raise ValueError(f"W4Weight.quantize: groups of 32, 64 or 128 that divide k; not {group} for {tuple(w.shape)}")
        if codes is None:
            codes = torch.empty(n, k // 2, dtype=torch.uint8, device=w.device)
        if scales is None:
            scales = torch.empty(n, k // group, dtype=torch.bfloat16, device=w.device)
        if codes.shape != (n, k // 2) or scales.shape != (n, k // group) or codes.device != w.device:
            raise ValueError("W4Weight.quantize: codes [n, k / 2] and scales [n, k / group] on w's device")
        q = cls(codes, scales)
        B.dec_w4_quantize(q._c, w.data_ptr(), w.stride(0) if n > 1 else k, _DT[w.dtype], _raw_stream(q._c.device))
        return q

    def dequantize(self, dtype: torch.dtype = torch.float32, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """The matrix that the codes and scales stand for, [n, k], as dtype (or into out, as its type; out's rows start at
        multiples of 16 bytes)."""
        if out is None:
            if dtype not in _DT:
                raise ValueError("W4Weight.dequantize: f32 or bf16")
            out = torch.empty(self.shape, dtype=dtype, device=self.device)
        elif out.shape != self.shape or out.dtype not in _DT or out.device != self.device or out.stride(1) != 1:
            raise ValueError("W4Weight.dequantize: out is f32 or bf16 [n, k] on the weight's device")
        B.dec_w4_dequantize(self._c, out.data_ptr(), out.stride(0) if self.shape[0] > 1 else self.shape[1], _DT[out.dtype],
                            _raw_stream(self._c.device))
        return out

    def linear(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None, norm: Optional[torch.Tensor] = None,
               eps: float = 1e-5, out: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None) -> torch.Tensor:
        """residual + W a for x [tokens, k] (f32 or bf16, its rows at multiples of 16 bytes): a = x, or with a gain `norm` [k]
        its RMSNorm.  The result [tokens, n] has dtype, by default x's; `out` may be the residual itself.  For many bf16 tokens
        a norm or an fp32 result doubles the products (both keep more than bf16's bits)."""
        return self._run(None, x, 0, residual, norm, eps, out, dtype)

    def glu(self, up: "W4Weight", x: torch.Tensor, act: str = "silu", norm: Optional[torch.Tensor] = None,
            eps: float = 1e-5, out: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None) -> torch.Tensor:
        """act(W a) * (up a), the first half of a gated feed-forward block; act "silu" or "gelu_tanh"; else like linear."""
        if act not in _ACT:
            raise ValueError(f"W4Weight.glu: act is one of {sorted(_ACT)}, not {act!r}")
        return self._run(up, x, _ACT[act], None, norm, eps, out, dtype)

    def _prepare(self, up, x, act, residual, norm, eps, out):
        # the checks and sizes that repeat with every call of the same shapes
        n, k = self.shape
        if x.dim() != 2 or x.shape[1] != k or x.dtype not in _DT or x.device != self.device or x.stride(1) != 1:
            raise ValueError(f"W4Weight: x is f32 or bf16 [tokens, {k}], columns side by side, on the weight's device")
        if up is not None and (up.shape != self.shape or up.group != self.group or up.device != self.device):
            raise ValueError("W4Weight.glu: gate and up have one shape, group and device")
        if norm is not None and (norm.shape != (k,) or norm.dtype not in _DT or norm.device != self.device
                                 or norm.stride(0) != 1):
            raise ValueError(f"W4Weight: norm is f32 or bf16 [{k}] on the weight's device")
        m = x.shape[0]
        for what, t in (("out", out), ("residual", residual)):
            if t is not None and (t.shape != (m, n) or t.dtype != out.dtype or t.dtype not in _DT or t.device != self.device
                                  or (n > 1 and t.stride(1) != 1)):
                raise ValueError(f"W4Weight: {what} is [{m}, {n}] of the result's type (f32 or bf16), columns side by side, "
                                 "on the weight's device")
        stride = lambda t, cols: 0 if t is None else t.stride(0) if m > 1 else cols   # noqa: E731
        c = B.dec_w4_call(x.data_ptr(), None if norm is None else norm.data_ptr(),
                          None if residual is None else residual.data_ptr(), out.data_ptr(), stride(x, k),
                          stride(residual, n), stride(out, n), m, _DT[x.dtype], 0 if norm is None else _DT[norm.dtype],
                          _DT[out.dtype], act, 0, eps, self._dev.err_ptr, None, 0)
        need = B.dec_w4_workspace(self._c, None if up is None else up._c, c) if m else 0
        if len(self._calls) >= 64:   # prompts come in any length
            self._calls.clear()
        return c, need

    def _run(self, up, x, act, residual, norm, eps, out, dtype):
        if torch.is_grad_enabled() and (x.requires_grad or norm is not None and norm.requires_grad
                                        or residual is not None and residual.requires_grad
                                        or out is not None and out.requires_grad):
            raise ValueError("W4Weight: no backward pass, and x, norm, residual or out requires a gradient (call it under "
                             "torch.no_grad, or detach them)")
        if out is None:
            out = torch.empty(x.shape[0], self.shape[0], dtype=x.dtype if dtype is None else dtype, device=x.device)
        elif dtype is not None and out.dtype != dtype:
            raise ValueError("W4Weight: out is not of dtype")
        dev = self._dev
        key = (x.shape, x.stride(), x.dtype, x.device, out.shape, out.stride(), out.dtype, out.device, act, eps,
               None if up is None else (up.shape, up.group, up.device),
               None if residual is None else (residual.shape, residual.stride(), residual.dtype, residual.device),
               None if norm is None else (norm.shape, norm.stride(), norm.dtype, norm.device))
        with self._lock:   # the call record is this thread's until the launch
            got = self._calls.get(key)
            if got is None:
                got = self._calls[key] = self._prepare(up, x, act, residual, norm, eps, out)
            c, need = got
            c.x, c.out = x.data_ptr(), out.data_ptr()
            if norm is not None:
                c.gain = norm.data_ptr()
            if residual is not None:
                c.residual = residual.data_ptr()
            stream = _raw_stream(dev.index)
            if need:   # from torch's allocator, which hands it on in the stream's order
                ws = torch.empty(need, dtype=torch.uint8, device=self.device)
                c.workspace, c.workspace_bytes = ws.data_ptr(), need
            if up is None:
                B.dec_w4_linear(self._c, c, stream)
            else:
                B.dec_w4_glu(self._c, up._c, c, stream)
        return out

    def check(self) -> None:
        """Wait for all work on the device so far, on whatever stream and in whatever graph, and raise DecError if a W4Weight
        call gave up a wait since the last check.  Not while any stream is being captured."""
        torch.cuda.synchronize(self.device)
        bits = int(self._dev.err.item())
        if bits:
            self._dev.err.zero_()
            torch.cuda.synchronize(self.device)   # a later call on another stream adds its bits after this
            raise B.DecError(B.DEC_E_DEVICE_FAULT, f"4-bit weights: a wait gave up (error word 0x{bits:x})")
