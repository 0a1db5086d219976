"""Products of so many tokens that their tiles fill the card: there a CTA has one row tile and two blocks of tokens."""
import pytest
import torch

import _w4 as R
from test_w4_gpu import DT, W, normal, run_glu, run_linear   # noqa: F401  (W is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m, n, k, group", [(4095, 1001, 1152, 64), (3900, 1100, 1120, 32), (4000, 1537, 128, 128), (3999, 2500, 32, 32),
                                            (2700, 2049, 160, 32), (2049, 2177, 384, 64), (1025, 4100, 640, 128),
                                            (700, 6144, 2176, 128), (4500, 1030, 256, 64)])
def test_linear(W, dtype, m, n, k, group):   # noqa: F811
    run_linear(W, m, n, k, group, dtype, norm=False, residual=True, seed=m)
    run_linear(W, m, n, k, group, dtype, norm=True, residual=False, seed=m)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("m, n, k, group", [(4095, 520, 640, 128), (3900, 515, 1120, 32), (2049, 1057, 32, 32), (1300, 1600, 384, 64),
                                            (257, 6200, 1152, 128)])
def test_glu(W, dtype, act, m, n, k, group):   # noqa: F811
    run_glu(W, m, n, k, group, dtype, True, act, seed=m)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m, n, k, group", [(2048, 2300, 4096, 128), (3900, 1100, 1120, 32)])
def test_repeats_bit_for_bit(W, dtype, m, n, k, group):   # noqa: F811
    a, b = W(*R.random_matrix(n, k, group, 1)), W(*R.random_matrix(n, k, group, 2))
    x = normal(m, k, seed=3, dtype=DT[dtype])
    first, both = a.linear(x), a.glu(b, x)
    for _ in range(12):
        assert torch.equal(a.linear(x), first) and torch.equal(a.glu(b, x), both)
    a.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_tokens_do_not_mix(W, dtype):   # noqa: F811
    """A token's result is the same beside others that are not finite."""
    m, n, k = 3900, 1100, 640
    w, up = W(*R.random_matrix(n, k, 64, 1)), W(*R.random_matrix(n, k, 64, 2))
    x = normal(m, k, seed=3, dtype=DT[dtype])
    bad = [0, 127, 128, 1000, 3899]
    keep = torch.ones(m, dtype=torch.bool, device="cuda")
    keep[bad] = False
    y, z = w.linear(x), w.glu(up, x)
    x[bad, 5] = float("nan")
    x[1000, 7] = float("inf")
    y2, z2 = w.linear(x), w.glu(up, x)
    assert torch.equal(y2[keep], y[keep]) and torch.equal(z2[keep], z[keep])
    assert torch.isnan(y2[[0, 127, 128, 3899]]).all() and not torch.isfinite(y2[1000]).any()


def test_rows_behind_and_strides(W):   # noqa: F811
    """Results into a part of a wider matrix leave the rest of it as it was."""
    m, n, k = 3900, 1100, 640
    w = W(*R.random_matrix(n, k, 64, 1))
    x = normal(m, k + 64, seed=3)[:, 64:]
    wide = torch.full((m + 3, n + 11), 7.0, device="cuda")
    w.linear(x, out=wide[:m, 5:5 + n])
    assert torch.equal(wide[:m, 5:5 + n], w.linear(x.contiguous()))
    assert (wide[m:] == 7.0).all() and (wide[:, :5] == 7.0).all() and (wide[:, 5 + n:] == 7.0).all()
