"""Shared by the tests of the 8-bit K/V cache: the definitions in 64 bits and random caches."""
from __future__ import annotations

import math

import torch

LOW, HIGH = -40, 60          # exponents a stored scale may take


def e4m3(x: torch.Tensor) -> torch.Tensor:
    """fp64 values rounded to e4m3 (nearest, ties to even) from the format's definition; NaN and over 448: NaN."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp_min(-6).double() - 3.0)
    y = torch.round(x / step) * step
    return torch.where(x.abs() <= 448, y, torch.full_like(y, math.nan))


def exponent(top: float) -> int:
    """The least e with top <= 448 * 2^e, within the range."""
    e = LOW
    while e < HIGH and top > 448.0 * 2.0 ** e:
        e += 1
    return e


class Store:
    """K or V as fp64 e4m3 values and exponents, on the CPU: [pages, heads, page, dim] and [pages, heads, blocks]."""

    def __init__(self, pages, heads, page, dim, block):
        self.x = torch.zeros(pages, heads, page, dim, dtype=torch.float64)
        self.e = torch.zeros(pages, heads, page // block, dtype=torch.int64)
        self.block = block

    def values(self, pages) -> torch.Tensor:
        """[heads, positions, dim] of one row's pages."""
        x = self.x[pages] * torch.exp2(self.e[pages].double()).repeat_interleave(self.block, 2)[..., None]
        return x.transpose(0, 1).flatten(1, 2)

    def append(self, pages, first: int, new: torch.Tensor):
        """new [tokens, heads, dim] fp64 at positions first, first + 1, ... (negative ones are dropped)."""
        n, page = new.shape[0], self.x.shape[2]
        lo, end = max(first, 0), first + n
        for b in range(lo // self.block, (end - 1) // self.block + 1 if end > lo else 0):
            p0, p1 = max(lo, b * self.block), min(end, (b + 1) * self.block)
            pid, off = int(pages[b * self.block // page]), b * self.block % page
            held = p0 - b * self.block
            for h in range(new.shape[1]):
                x = new[p0 - first:p1 - first, h]
                fin = x[torch.isfinite(x)].abs()
                e = exponent(float(fin.max()) if fin.numel() else 0.0)
                was = int(self.e[pid, h, off // self.block])
                if held:
                    e = max(e, was)
                    old = self.x[pid, h, off:off + held]
                    if e > was:
                        self.x[pid, h, off:off + held] = e4m3(old * 2.0 ** (was - e))
                self.x[pid, h, off + held:off + held + p1 - p0] = e4m3(x * 2.0 ** -e)
                self.e[pid, h, off // self.block] = e

    def bytes(self):
        return self.x.float().to(torch.float8_e4m3fn).view(torch.uint8), (self.e + 127).to(torch.uint8)


def random_store(pages, heads, page, dim, block, g, spread=3):
    s = Store(pages, heads, page, dim, block)
    s.x = (torch.randn(s.x.shape, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn).double()
    s.e = torch.randint(-7 - spread, -5 + spread, s.e.shape, generator=g)
    return s


def table_of(rows, per_row, g):
    return torch.randperm(rows * per_row + 3, generator=g)[:rows * per_row].view(rows, per_row).int()


def sees(p, length, window, sinks):
    """[tokens, positions] of what tokens at positions p see."""
    j = torch.arange(length)[None, :]
    p = p[:, None]
    m = j <= p
    if window:
        m &= (j > p - window) | (j < sinks)
    return m


def attend(q, k, v, p, window=0, sinks=0, scale=None):
    """One row: q [tokens, heads, dim], k, v [kv_heads, positions, dim], all fp64; p the tokens' positions.
    Returns (out, sum p |v|, sum |q k| * scale at most): the result and what its error is measured by."""
    n, hq, d = q.shape
    g = hq // k.shape[0]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    m = sees(p, k.shape[1], window, sinks)
    out, mass, score = torch.zeros_like(q), torch.zeros_like(q), 0.0
    for a in range(hq):
        kk, vv = k[a // g], v[a // g]
        s = (q[:, a] @ kk.T) * scale
        s = torch.where(m, s, torch.full_like(s, -math.inf))
        top = s.amax(1, keepdim=True)
        w = torch.where(m, torch.exp(s - torch.where(top > -math.inf, top, torch.zeros_like(top))), torch.zeros_like(s))
        l = w.sum(1, keepdim=True)
        w = torch.where(m, w / torch.where(l == 0, torch.ones_like(l), l), torch.zeros_like(w))
        # what is not seen does not reach the result, whatever it holds
        for t in range(n):
            at = m[t]
            if at.any():
                out[t, a] = w[t, at] @ vv[at]
                mass[t, a] = w[t, at] @ vv[at].abs()
        seen = kk[m.any(0)]
        if seen.numel():
            score = max(score, float((q[:, a].abs() @ seen.abs().T).nan_to_num(0.0).max()) * scale)
    return out, mass, score


def bound(mass, score, out, dtype, dim, n):
    """What an attention result may be off: relative to sum p |v|,
      a score's error d = score * (dim * 2^-24 [fp32 sums of dim products] + 2^-20 [q in two f16 parts, scale factors])
      moves each weight, and their sum, by d; the exponential and its argument (at most score * log2 e below the
      maximum, in fp32) by 2^-21 + 3 * score * 2^-24 each; fp32 sums over n positions by sqrt(n) * 2^-23;
      f16 weights (bf16 q only) by 2^-11;
    and the result's own rounding (bf16 2^-8, fp32 2^-24) relative to itself."""
    rel = 2 * score * (dim * 2.0 ** -24 + 2.0 ** -20) + 2 * (2.0 ** -21 + 3 * score * 2.0 ** -24) + math.sqrt(n) * 2.0 ** -23
    rel += 2.0 ** -11 if dtype == torch.bfloat16 else 0.0
    return rel * mass + out.abs() * (torch.finfo(dtype).eps / 2) + 1e-30
