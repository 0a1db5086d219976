"""The 4-bit weights without a GPU: what their calls refuse, before any device call, and the tests' own definitions."""
import ctypes
import math

import pytest
import torch

import _w4 as R


@pytest.fixture(scope="module")
def B():
    from graph_replay_gb300 import build, _binding
    build.build()
    return _binding


PTR = 1 << 20   # a 256-byte aligned address that is never read: the checks come first


def weight(B, **kw):
    w = dict(codes=PTR, scales=PTR, n=64, k=256, group=64, device=0)
    w.update(kw)
    return B.dec_w4_weight(**w)


def call(B, **kw):
    c = dict(x=PTR, gain=None, residual=None, out=PTR + (1 << 18), x_stride=256, residual_stride=0, out_stride=64, tokens=3, x_dtype=0,
             gain_dtype=0, out_dtype=0, act=0, reserved=0, eps=1e-5, err=PTR, workspace=None, workspace_bytes=0)
    c.update(kw)
    return B.dec_w4_call(**c)


WEIGHTS = [(dict(codes=None), 1, "codes"), (dict(scales=None), 1, "scales"), (dict(codes=PTR + 8), 1, "aligned"),
           (dict(scales=PTR + 1), 1, "aligned"), (dict(n=0), 1, "n and k"), (dict(k=0), 1, "n and k"), (dict(n=-5), 1, "n and k"),
           (dict(group=16), 2, "group"), (dict(group=0), 2, "group"), (dict(k=96, group=64), 1, "multiple"),
           (dict(k=1 << 21), 2, "2^20"), (dict(n=1 << 20, k=1 << 15), 2, "2^33"), (dict(device=-1), 1, "device")]


@pytest.mark.parametrize("what, code, word", WEIGHTS)
def test_bad_weights(B, what, code, word):
    w, size = weight(B, **what), ctypes.c_size_t()
    lib = B.lib()
    for rc in (lib.dec_w4_linear(w, call(B), None), lib.dec_w4_glu(weight(B), w, call(B), None), lib.dec_w4_glu(w, weight(B), call(B), None),
               lib.dec_w4_quantize(w, PTR, 256, 0, None), lib.dec_w4_dequantize(w, PTR, 256, 0, None),
               lib.dec_w4_workspace(w, None, call(B), size)):
        assert rc == code and word in B.last_error(None)


@pytest.mark.parametrize("what, code, word", [
    (dict(tokens=-1), 1, "tokens"), (dict(x=None), 1, "x"), (dict(x=PTR + 4), 1, "x"), (dict(x_stride=252), 1, "x"),
    (dict(x_stride=258), 1, "x"), (dict(x_stride=-256), 1, "x"), (dict(out=None), 1, "out"), (dict(out=PTR + 2), 1, "out"),
    (dict(out_stride=63), 1, "out"), (dict(x_dtype=2), 1, "x_dtype"), (dict(out_dtype=7), 1, "out_dtype"),
    (dict(gain=PTR, gain_dtype=2), 1, "gain"), (dict(gain=PTR + 8), 1, "gain"), (dict(gain=PTR, eps=-1.0), 1, "eps"),
    (dict(gain=PTR, eps=math.nan), 1, "eps"), (dict(gain=PTR, eps=1e300), 1, "eps"), (dict(err=None), 1, "err"),
    (dict(err=PTR + 2), 1, "err"), (dict(tokens=1 << 26), 2, "tokens"), (dict(tokens=(1 << 21) + 1), 2, "tokens"),
    (dict(out=PTR), 1, "overlaps"), (dict(out=PTR + 1024), 1, "overlaps"), (dict(out=PTR + 4 * 255, out_stride=256), 1, "overlaps"),
    (dict(out=PTR - 4 * 62, out_stride=256), 1, "overlaps"), (dict(gain=PTR + (1 << 16), out=PTR + (1 << 16) + 64), 1, "overlaps")])
def test_bad_calls(B, what, code, word):
    lib = B.lib()
    for rc in (lib.dec_w4_linear(weight(B), call(B, **what), None), lib.dec_w4_glu(weight(B), weight(B), call(B, **what), None)):
        assert rc == code and word in B.last_error(None)


def test_bad_residuals_activations_and_pairs(B):
    lib = B.lib()
    for what, word in ((dict(residual=PTR + 1, residual_stride=64), "residual"), (dict(residual=PTR, residual_stride=60), "residual"),
                       (dict(residual=PTR + (1 << 18), residual_stride=128), "stride"),
                       (dict(residual=PTR + (1 << 18) + 4, residual_stride=64), "overlaps")):
        assert lib.dec_w4_linear(weight(B), call(B, **what), None) == 1 and word in B.last_error(None)
    assert lib.dec_w4_glu(weight(B), weight(B), call(B, residual=PTR + 4096, residual_stride=64), None) == 1
    assert "residual" in B.last_error(None)
    assert lib.dec_w4_glu(weight(B), weight(B), call(B, act=2), None) == 1 and "act" in B.last_error(None)
    for kw in (dict(n=128), dict(k=512), dict(group=32), dict(device=1)):
        assert lib.dec_w4_glu(weight(B), weight(B, **kw), call(B), None) == 1 and "one shape" in B.last_error(None)
    assert lib.dec_w4_glu(weight(B), None, call(B), None) == 1 and "up" in B.last_error(None)
    assert lib.dec_w4_linear(None, call(B), None) == 1 and lib.dec_w4_linear(weight(B), None, None) == 1
    assert lib.dec_w4_workspace(weight(B), None, call(B), None) == 1


def test_bad_storing(B):
    lib = B.lib()
    for rc in (lib.dec_w4_quantize(weight(B), None, 256, 0, None), lib.dec_w4_quantize(weight(B), PTR + 4, 256, 0, None),
               lib.dec_w4_quantize(weight(B), PTR, 255, 0, None), lib.dec_w4_quantize(weight(B), PTR, 256, 2, None),
               lib.dec_w4_dequantize(weight(B), None, 256, 1, None), lib.dec_w4_dequantize(weight(B), PTR, 260, 1, None)):
        assert rc == 1


def test_columns_of_one_wider_matrix_do_not_overlap(B):
    """x and out side by side in rows of 1024 floats, either way round: refused for nothing but the device that is not there."""
    lib = B.lib()
    for x, out in ((PTR, PTR + 1024), (PTR + 1024, PTR + 256), (PTR + 4096 * 2, PTR + 1024)):
        c = call(B, x=x, x_stride=1024, out=out, out_stride=1024, eps=0.0)
        if not torch.cuda.is_available():
            assert lib.dec_w4_linear(weight(B), c, None) == 5   # DEC_E_CUDA: every check before it passed


def test_no_tokens_is_nothing_to_do(B):
    size = ctypes.c_size_t(7)
    assert B.lib().dec_w4_linear(weight(B), call(B, tokens=0, x=None, out=None), None) == 0
    assert B.lib().dec_w4_workspace(weight(B), None, call(B, tokens=0), size) == 0 and size.value == 0


# ---- the definitions that the GPU tests use ----

def test_codes_and_bytes():
    q = torch.arange(-8, 8).view(1, 16).double()
    b = R.pack(q)
    assert b.tolist() == [[0x98, 0xBA, 0xDC, 0xFE, 0x10, 0x32, 0x54, 0x76]]
    assert torch.equal(R.codes_of(b), q)


def test_rounding_to_bf16():
    x = torch.randn(4000, dtype=torch.float64) * torch.exp2(torch.randint(-30, 30, (4000,)).double())
    assert torch.equal(R.to_bf16(x), x.float().bfloat16().double()) or \
        (R.to_bf16(x) != x.float().bfloat16().double()).sum() <= 1   # fp32 first may round a value onto a border
    tie = torch.tensor([1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8], dtype=torch.float64)
    assert R.to_bf16(tie).tolist() == [1.0, 1 + 2.0 ** -6]


def test_quantize_definition():
    w = torch.zeros(1, 64)
    w[0, 0], w[0, 1], w[0, 2], w[0, 3], w[0, 40] = 7.0, 0.5, 1.5, -2.4, 2.0 ** -120
    q, s = R.quantize(w, 32)
    assert s.tolist() == [[1.0, 0.0]] and q[0, :4].tolist() == [7.0, 0.0, 2.0, -2.0] and q[0, 40] == 0
    w[0, 41] = math.inf
    assert math.isnan(R.quantize(w, 32)[1][0, 1])


def test_plain_forms_agree():
    """The measured plain form and the tests' definition store the same bytes."""
    import perf.more_operators as M
    w = torch.randn(20, 256) * torch.exp(torch.randn(20, 1))
    for group in (32, 64, 128):
        c, s = M.plain_quantize(w, group)
        q, t = R.quantize(w, group)
        assert torch.equal(R.codes_of(c), q) and torch.equal(s.double(), t)
        assert torch.equal(M.plain_values(c, s).double(), R.values(c, s))


def test_activations_of_the_block():
    g, u = torch.tensor([0.0, 1.0, -30.0, 30.0], dtype=torch.float64), torch.full((4,), 2.0, dtype=torch.float64)
    assert torch.allclose(R.glu("silu", g, u), torch.nn.functional.silu(g) * u, atol=1e-12)
    assert torch.allclose(R.glu("gelu_tanh", g, u), torch.nn.functional.gelu(g, approximate="tanh") * u, atol=1e-12)
