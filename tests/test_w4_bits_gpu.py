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
        other = int((got.double() != R.to_bf16(want)).sum())
        assert other <= max(1, OTHER * got.numel()), f"{what}: {other} of {got.numel()} results are others"


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


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m", [1, 3, 8, 11, 24, 300])
def test_sizes_at_both_ends(W, m, group, dtype):   # noqa: F811
    """Activations from 2^-110 to 2^123 and scales that bring their products back: no step leaves fp32's range where the result
    does not."""
    n, k = 70, 2176
    codes, _ = R.random_matrix(n, k, group, 5)
    row = torch.arange(n, device="cuda")[:, None]
    x = normal(m, k, seed=1)
    tok = torch.arange(m, device="cuda")[:, None]
    for up, down in ((120, -40), (123, -110), (-100, 40), (-90, 110), (60, -100)):
        s = (torch.rand(n, k // group, device="cuda") + 0.5) * torch.exp2(down + (row % 3).float())
        far = (x * torch.exp2(torch.where(tok % 2 == 0, float(up), float(-down)))).to(DT[dtype])
        w = W(codes, s.bfloat16())
        want = far.double() @ R.values(codes, w.scales).T
        got = w.linear(far, dtype=torch.float32)
        for t in range(m):
            err = (got[t].double() - want[t]).norm()
            assert err <= KEPT * want[t].norm(), f"2^{up}, 2^{down}, token {t}: {err / want[t].norm():.3g}"
    w.check()


def test_one_large_block_of_columns(W):   # noqa: F811
    """A token whose large values lie in one block of columns, and tokens beside it that have none: theirs stay as they are."""
    n, k = 300, 4096
    a = R.random_matrix(n, k, 64, 5)
    w = W(a[0], (a[1].float() * 2.0 ** -30).bfloat16())
    x = normal(6, k, seed=2)
    alone = w.linear(x)
    x[2, 1500:1510] = 1e38
    x[4, 100] = -3e38
    got = w.linear(x)
    want = x.double() @ R.values(w.codes, w.scales).T
    keep = [0, 1, 3, 5]
    assert torch.equal(got[keep], alone[keep])
    for t in range(6):
        assert (got[t].double() - want[t]).norm() <= KEPT * want[t].norm()
    w.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m", [1, 8, 20])
def test_largest_sums(W, m, dtype):   # noqa: F811
    """The largest activations and codes, all of one sign: 128 columns make 2^138."""
    n, k = 40, 1024
    codes = torch.full((n, k // 2), 0x88, dtype=torch.uint8, device="cuda")
    for group in (32, 64, 128):
        w = W(codes, torch.full((n, k // group), 2.0 ** -20, dtype=torch.bfloat16, device="cuda"))
        x = torch.full((m, k), torch.finfo(DT[dtype]).max, device="cuda", dtype=DT[dtype])
        got = w.linear(x, dtype=torch.float32)
        want = x[0, 0].double() * -8.0 * k * 2.0 ** -20
        assert ((got.double() - want).abs() <= KEPT * want.abs()).all()
    w.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 2, 31, 33, 63, 65, 97, 127, 129, 255, 257])
def test_rows_that_do_not_fill_a_warp(W, n, dtype):   # noqa: F811
    """Many tokens: lanes without an output row write nothing, and read the sums with the others all the same."""
    for m, k in ((20, 256), (100, 384), (4000, 128)):
        a, b, x = inputs(m, n, k, 64, DT[dtype], n)
        w, u, h = W(*a), W(*b), normal(m, n, seed=n + 5, dtype=DT[dtype])
        y, z = x.double() @ R.values(*a).T, x.double() @ R.values(*b).T
        check(w.linear(x, residual=h), y + h.double(), "linear")
        check(w.glu(u, x, act="gelu_tanh"), R.glu("gelu_tanh", y, z), "glu")
    w.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m", [1, 3, 8, 20, 130])
def test_normed_tokens_of_far_sizes(W, m, dtype):   # noqa: F811
    """From 2^-58 to 2^55, the sum of squares within fp32; with no eps the sizes go out again."""
    n, k = 70, 2176
    a, _, x = inputs(m, n, k, 64, torch.float32, 3)
    size = torch.tensor([55.0, 0.0, -58.0], device="cuda")[torch.arange(m, device="cuda") % 3]
    x = (x * torch.exp2(size)[:, None]).to(DT[dtype])
    gain = (1.0 + 0.3 * normal(k, seed=9)).to(DT[dtype])
    w = W(*a)
    for eps in (0.0, 1e-5):
        want = R.activation(x, gain, eps) @ R.values(*a).T
        got = w.linear(x, norm=gain, eps=eps, dtype=torch.float32)
        assert ((got.double() - want).norm(dim=1) <= KEPT * want.norm(dim=1)).all(), eps
    w.check()
