"""The 4-bit weights against their definitions in 64 bits."""
import math

import pytest
import torch

import _w4 as R

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def W():
    from graph_replay_gb300 import W4Weight, build
    build.build()
    return W4Weight


def normal(*shape, seed=0, dtype=torch.float32):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


# ---- storing ----

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n, k", [(1, 128), (3, 384), (129, 1152), (1000, 4096)])
def test_store(W, dtype, group, n, k):
    w = normal(n, k, seed=n, dtype=DT[dtype]) * 0.02
    got = W.quantize(w, group)
    q, s = R.quantize(w, group)
    assert torch.equal(got.scales.double(), s)
    assert torch.equal(R.codes_of(got.codes), q)
    v = R.values(got.codes, got.scales)
    assert torch.equal(got.dequantize().double(), v)
    assert torch.equal(got.dequantize(torch.bfloat16).double(), R.to_bf16(v))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_store_ties_and_neighbours(W, dtype):
    # one group a scale; values at and next to the borders (j + 1/2) * scale between codes
    rows = []
    g = torch.Generator().manual_seed(3)
    for i in range(64):
        s = float(torch.rand((), generator=g) + 1.0) * 2.0 ** int(torch.randint(-40, 40, (), generator=g))
        s = float(torch.tensor(s).bfloat16())
        top = torch.tensor([7.0 * s], dtype=torch.float64)
        mid = (torch.arange(-7, 7).double() + 0.5) * s
        near = torch.cat([mid, torch.nextafter(mid.float(), torch.tensor(math.inf)).double(),
                          torch.nextafter(mid.float(), torch.tensor(-math.inf)).double()])
        row = torch.cat([top, near, torch.zeros(64 - 1 - near.numel(), dtype=torch.float64)])
        rows.append(row)
    w = torch.stack(rows).to(DT[dtype]).cuda()
    got = W.quantize(w, 64)
    q, s = R.quantize(w, 64)
    assert torch.equal(got.scales.double(), s) and torch.equal(R.codes_of(got.codes), q)


def test_store_extremes(W):
    w = normal(8, 256, seed=1)
    w[0] = 0.0
    w[1] = 2.0 ** -140
    w[2] *= 1e37
    w[3, 5] = math.nan
    w[3, 200] = math.inf
    w[4, 128:] = -math.inf
    w[5] = 3.4e38
    w[6] *= 7 * 2.0 ** -100
    got = W.quantize(w, 128)
    q, s = R.quantize(w, 128)
    assert torch.equal(torch.isnan(got.scales), torch.isnan(s))
    assert torch.equal(got.scales.double().nan_to_num(), s.nan_to_num())
    assert torch.equal(R.codes_of(got.codes), q)
    v = got.dequantize()
    assert torch.isnan(v[3]).all() and torch.isnan(v[4, 128:]).all() and not torch.isnan(v[[0, 1, 2, 5, 6, 7]]).any()


def test_store_strided_rows(W):
    big = normal(40, 1024, seed=5)
    w = big[:, 256:640]
    got = W.quantize(w, 64)
    assert torch.equal(got.codes, W.quantize(w.contiguous(), 64).codes)
    out = torch.full((40, 512), 7.0, device="cuda")
    got.dequantize(out=out[:, 64:448])
    assert torch.equal(out[:, 64:448].double(), R.values(got.codes, got.scales))
    assert (out[:, :64] == 7.0).all() and (out[:, 448:] == 7.0).all()


# ---- the linear layer ----

def run_linear(W, m, n, k, group, dtype, norm, residual, seed=0, out_dtype=None, x=None):
    codes, scales = R.random_matrix(n, k, group, seed)
    w = W(codes, scales)
    dt = DT[dtype]
    if x is None:
        x = (normal(m, k, seed=seed + 1) * torch.exp(normal(m, 1, seed=seed + 2))).to(dt)
    gain = (1.0 + 0.2 * normal(k, seed=seed + 3)).to(dt) if norm else None
    od = out_dtype or dt
    res = normal(m, n, seed=seed + 4, dtype=od) if residual else None
    got = w.linear(x, residual=res, norm=gain, dtype=od)
    a = R.activation(x, gain, 1e-5)
    v = R.values(codes, scales)
    want = a @ v.T
    bits = 21 if dtype == "f32" or (norm and m <= 8) else 11 if norm else 40
    bound = R.product_bound(a, v, bits, k) + (R.EPS[torch.float32] * 4 * want.abs())
    if residual:
        want = want + res.double()
        bound = bound + 2.0 ** -24 * want.abs()
    if od == torch.float32 and dtype == "f32" and want.numel() > 500:
        # the bound is the worst case; steps of 2^-23 that go either way add to a few 2^-21 of the whole
        assert (got.double() - want).norm() <= 2.0 ** -18 * want.norm()
    w.check()
    return R.close(got, want, bound, f"linear {m}x{n}x{k}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m, n, k", [(1, 1, 128), (1, 48, 256), (2, 100, 1152), (3, 1001, 1152), (4, 513, 2048), (5, 64, 384),
                                     (8, 2048, 2048), (8, 130, 14336), (1, 4096, 14336), (7, 31, 16384)])
def test_linear_few_tokens(W, dtype, group, m, n, k):
    run_linear(W, m, n, k, group, dtype, norm=False, residual=False, seed=m + n)
    run_linear(W, m, n, k, group, dtype, norm=True, residual=True, seed=m + n)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m, n, k, group", [(9, 200, 256, 64), (16, 1000, 1120, 32), (17, 300, 2048, 128), (33, 129, 4096, 32),
                                            (64, 640, 1024, 64), (100, 513, 4096, 128), (257, 250, 640, 128),
                                            (1000, 384, 1152, 64), (40, 64, 14336, 128)])
def test_linear_many_tokens(W, dtype, m, n, k, group):
    run_linear(W, m, n, k, group, dtype, norm=False, residual=True, seed=m)
    run_linear(W, m, n, k, group, dtype, norm=True, residual=False, seed=m)


# ---- the gated block ----

def run_glu(W, m, n, k, group, dtype, norm, act, seed=0):
    gc, gs = R.random_matrix(n, k, group, seed)
    uc, us = R.random_matrix(n, k, group, seed + 9)
    dt = DT[dtype]
    x = (normal(m, k, seed=seed + 1) * torch.exp(normal(m, 1, seed=seed + 2))).to(dt)
    gain = (1.0 + 0.2 * normal(k, seed=seed + 3)).to(dt) if norm else None
    gate, up = W(gc, gs), W(uc, us)
    got = gate.glu(up, x, act=act, norm=gain)
    a = R.activation(x, gain, 1e-5)
    gv, uv = R.values(gc, gs), R.values(uc, us)
    g, u = a @ gv.T, a @ uv.T
    bits = 21 if dtype == "f32" or (norm and m <= 8) else 11 if norm else 40
    bg, bu = R.product_bound(a, gv, bits, k) + 2.0 ** -22 * g.abs(), R.product_bound(a, uv, bits, k) + 2.0 ** -22 * u.abs()
    # both functions have a slope of at most 1.13 in size; their own rounding is a few steps of fp32 (the exponent of
    # gelu_tanh turns a relative step of z into |2 z| of the result, and beyond |z| = 50 the result is 0 or g)
    want = R.glu(act, g, u)
    own = (2.0 ** -21 * torch.clamp(1 + 4 * g.abs() ** 3, max=100.0)) * (g * u).abs()
    bound = 1.13 * bg * (u.abs() + bu) + bu * torch.maximum(R.glu(act, g, torch.ones_like(g)).abs(), 0.2 * torch.ones_like(g)) + own
    gate.check()
    return R.close(got, want, bound, f"glu {m}x{n}x{k}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("m, n, k, group", [(1, 1, 128, 128), (1, 100, 1152, 32), (3, 257, 2048, 64), (8, 1001, 4096, 32),
                                            (8, 64, 14336, 128), (17, 130, 1120, 32), (100, 300, 2048, 128),
                                            (300, 129, 640, 64)])
def test_glu(W, dtype, act, m, n, k, group):
    run_glu(W, m, n, k, group, dtype, True, act, seed=m)
    run_glu(W, m, n, k, group, dtype, False, act, seed=m + 1)


@pytest.mark.parametrize("m, n, k, group, dtype", [(40, 6144, 4096, 128, "bf16"), (64, 4096, 14336, 64, "f32"), (9, 513, 4096, 32, "f32"),
                                                   (300, 2000, 2048, 128, "f32"), (8, 4096, 14336, 128, "f32"), (3, 1001, 1120, 32, "bf16"),
                                                   (1000, 1536, 1152, 64, "bf16")])
def test_repeats_bit_for_bit(W, m, n, k, group, dtype):
    """Results do not depend on when copies land: 40 calls in a row, with other work between, give the same bits."""
    a, b = W(*R.random_matrix(n, k, group, 1)), W(*R.random_matrix(n, k, group, 2))
    x = normal(m, k, seed=3, dtype=DT[dtype])
    first, both = a.linear(x), a.glu(b, x)
    run = R.activation(x, None, 0.0) @ R.values(a.codes, a.scales).T
    R.close(first, run, R.product_bound(x.double(), R.values(a.codes, a.scales), 21 if dtype == "f32" else 40, k), "linear")
    other = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    for i in range(40):
        if i % 4 == 0:
            other.fill_(i)     # the weights leave the cache
        assert torch.equal(a.linear(x), first) and torch.equal(a.glu(b, x), both), i
    a.check()
