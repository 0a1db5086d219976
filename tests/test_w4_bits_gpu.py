"""How many bits the products with 4-bit weights keep: the same in a prompt as in a step, whatever the activations' type."""
import pytest
import torch

import _w4 as R
from test_w4_gpu import DT, W, normal   # noqa: F401  (W is a fixture)

pytestmark = pytest.mark.gpu

# Activations enter to 2^-22 of themselves (in full without a norm, where they are bf16), a sum of 256 columns loses at most 16
# cuts of 2^-23 and is then added with rounding: about 2^-20 of the whole, in unlike directions from sum to sum.
KEPT = 2.0 ** -18
# A bf16 result is another than the exact value's only where a border between two lies as near as KEPT of the results' size: for
# a result of that size twice in 2^10 (steps of 2^-8), and for one 2^j times smaller, of which there are 2^j times fewer, 2^j
# times as often; nine such sizes count.
OTHER = 0.02


def check(got, want, what=""):
    err = (got.double() - want).norm() / want.norm()
    if got.dtype == torch.float32:
        assert err <= KEPT, f"{what}: off by {err:.3g} of the whole"
    else:
        other = (got.double() != R.to_bf16(want)).double().mean().item()
        assert other <= OTHER, f"{what}: {other:.3g} of the results are others"


def inputs(m, n, k, group, dtype, seed):
    x = (normal(m, k, seed=seed) * torch.exp(0.5 * normal(m, 1, seed=seed + 1))).to(dtype)
    return R.random_matrix(n, k, group, seed + 2), R.random_matrix(n, k, group, seed + 3), x


@pytest.mark.parametrize("gain_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("m, n, k, group", [(4, 600, 2048, 64), (8, 300, 4096, 128), (9, 300, 4096, 128), (40, 1000, 4096, 32), (129, 513, 1120, 32),
                                            (1000, 640, 2048, 128), (3000, 1100, 640, 64)])
def test_normed_bf16_tokens(W, m, n, k, group, out, gain_dtype):   # noqa: F811
    """The norm's product with a gain has more than bf16's bits."""
    a, b, x = inputs(m, n, k, group, torch.bfloat16, m)
    gain = (1.0 + 0.3 * normal(k, seed=9)).to(DT[gain_dtype])
    w, u = W(*a), W(*b)
    act = R.activation(x, gain, 1e-5)
    y, z = act @ R.values(*a).T, act @ R.values(*b).T
    check(w.linear(x, norm=gain, dtype=DT[out]), y, "linear")
    check(w.glu(u, x, norm=gain, dtype=DT[out]), R.glu("silu", y, z), "glu")
    w.check()


@pytest.mark.parametrize("m, n, k, group", [(16, 300, 14336, 128), (17, 300, 14336, 128), (64, 513, 14336, 64), (300, 256, 14336, 32),
                                            (1000, 640, 4096, 128), (4095, 1100, 14336, 128), (40, 64, 1 << 18, 128)])
def test_fp32_results_of_bf16_tokens(W, m, n, k, group):   # noqa: F811
    """What the tensor cores cut off does not add up over the columns."""
    a, b, x = inputs(m, n, k, group, torch.bfloat16, m)
    w, u = W(*a), W(*b)
    y, z = x.double() @ R.values(*a).T, x.double() @ R.values(*b).T
    check(w.linear(x, dtype=torch.float32), y, "linear")
    check(w.glu(u, x, dtype=torch.float32), R.glu("silu", y, z), "glu")
    w.check()


@pytest.mark.parametrize("m, n, k", [(20, 200, 1 << 16), (40, 64, 1 << 18), (200, 30, 1 << 20)])
def test_bf16_results_over_many_columns(W, m, n, k):   # noqa: F811
    a, _, x = inputs(m, n, k, 128, torch.bfloat16, m)
    w = W(*a)
    check(w.linear(x), x.double() @ R.values(*a).T, "linear")
    w.check()
