"""Shared by the tests of the 4-bit weights: the definitions in 64 bits, random matrices, and how far results may be off."""
from __future__ import annotations

import math

import torch

EPS = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}   # half a step, relative to the value


def to_bf16(x: torch.Tensor) -> torch.Tensor:
    """fp64 values to 8 significant bits, to the nearest, ties to even."""
    b = x.contiguous().view(torch.int64)
    return (((b + (2 ** 44 - 1) + ((b >> 45) & 1)) >> 45) << 45).view(torch.float64)


def quantize(w: torch.Tensor, group: int):
    """(codes as whole numbers [n, k], scales [n, k / group]) of w, all fp64."""
    x = w.double().unflatten(1, (-1, group))
    bad = ~torch.isfinite(x).all(-1)
    top = torch.where(torch.isfinite(x), x, 0.0).abs().amax(-1)
    s = to_bf16(top / torch.full((), 7.0, dtype=torch.float64, device=w.device))
    s = torch.where(s < 2.0 ** -100, 0.0, s)
    q = torch.round(torch.where((s > 0)[..., None], x, 0.0) / torch.where(s > 0, s, 1.0)[..., None])
    q = torch.where(bad[..., None], 0.0, q)
    return q.flatten(1), torch.where(bad, math.nan, s)


def pack(q: torch.Tensor) -> torch.Tensor:
    """Whole numbers -8 .. 7 [n, k] as the stored bytes."""
    b = q.long() & 15
    return (b[:, 0::2] | (b[:, 1::2] << 4)).to(torch.uint8)


def codes_of(b: torch.Tensor) -> torch.Tensor:
    """The whole numbers that stored bytes hold, fp64."""
    b = b.long()
    q = torch.stack([b & 15, b >> 4], -1).flatten(1)
    return (q - 16 * (q >= 8).long()).double()


def values(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """The fp64 matrix of stored bytes and scales."""
    q = codes_of(codes)
    return (q.unflatten(1, (scales.shape[1], -1)) * scales.double()[..., None]).flatten(1)


def random_matrix(n, k, group, seed=0, device="cuda", low=-8, spread=0.5):
    """(bytes, scales): any codes, scales of unlike size."""
    g = torch.Generator(device).manual_seed(seed)
    q = torch.randint(low, 8, (n, k), generator=g, device=device)
    s = 0.01 * torch.exp(spread * torch.randn(n, k // group, generator=g, device=device))
    return pack(q), s.to(torch.bfloat16)


def activation(x, norm, eps):
    """The fp64 activations of a call."""
    x = x.double()
    if norm is None:
        return x
    return x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * norm.double()


def glu(act, g, u):
    if act == "silu":
        return g * torch.sigmoid(g) * u
    z = math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)
    return g * torch.sigmoid(2.0 * z) * u


def product_bound(a, w, part_bits, k):
    """How far a product sum_k w a may be off: each activation enters to 2^-part_bits of itself (or 2^-39 of the largest
    beside it), and fp32 sums lose at most 2^-23 of the absolute values' sum a step (the tensor core cuts off).  Steps: one
    for each 16 columns where activations are one part; with two, 16 before the sums of both are taken over and rounded, each
    256 columns.  A few more join warps and splits."""
    mag = a.abs() @ w.abs().T
    top = a.abs().amax(-1, keepdim=True) * w.abs().sum(-1)[None]
    steps = 64 + k // 256 if part_bits == 21 else k // 16 + 24
    return mag * (2.0 ** -part_bits + steps * 2.0 ** -23) + top * 2.0 ** -38


def close(got, want, bound, what=""):
    """|got - want| within the result's rounding and the bound before it."""
    tol = EPS[got.dtype] * (want.abs() + bound) * 1.0001 + bound + 2.0 ** -140
    err = (got.double() - want).abs()
    assert not torch.isnan(got).any(), f"{what}: NaN"
    worst = (err / tol).max().item() if err.numel() else 0.0
    assert worst <= 1.0, f"{what}: off by {worst:.3g} of what is allowed"
    return worst
