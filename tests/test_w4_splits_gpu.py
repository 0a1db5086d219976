"""Products whose columns are shared by a cluster's CTAs in unequal parts: 128 columns at a time do not divide evenly."""
import pytest

from test_w4_gpu import W, run_glu, run_linear   # noqa: F401  (W is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m, n, k, group", [(7, 1, 15040, 64), (8, 200, 14464, 64), (8, 4096, 14464, 128), (5, 33, 12960, 32), (8, 64, 9856, 128),
                                            (4, 1000, 16256, 64), (3, 17, 16320, 64), (8, 512, 10368, 128), (6, 300, 7296, 128),
                                            (16, 40, 15040, 32)])
def test_few_tokens(W, dtype, m, n, k, group):   # noqa: F811
    for norm in (False, True):
        run_linear(W, m, n, k, group, dtype, norm=norm, residual=norm, seed=m + n)
        run_glu(W, m, n, k, group, dtype, norm, "silu" if norm else "gelu_tanh", seed=m + n)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m, n, k, group", [(20, 1, 15040, 64), (40, 300, 14464, 128), (17, 1000, 2432, 128), (64, 513, 4480, 64),
                                            (100, 70, 10400, 32), (33, 4096, 1184, 32)])
def test_more_tokens(W, dtype, m, n, k, group):   # noqa: F811
    for norm in (False, True):
        run_linear(W, m, n, k, group, dtype, norm=norm, residual=norm, seed=m + n)
        run_glu(W, m, n, k, group, dtype, norm, "silu" if norm else "gelu_tanh", seed=m + n)


@pytest.mark.parametrize("tokens", [8, 7, 5, 3, 2, 1])
@pytest.mark.parametrize("chunks", range(97, 128, 5))
def test_every_remainder(W, tokens, chunks):   # noqa: F811
    k = 128 * chunks - 64 * (chunks % 2)
    run_linear(W, tokens, 90, k, 64, "f32", norm=True, residual=True, seed=chunks)
    run_glu(W, tokens, 90, k, 64, "f32", True, "silu", seed=chunks)
