"""Attention over the 8-bit K/V cache where softmax weights, and the scales of V's blocks, lie far apart: the definition
in 64 bits holds relative to sum p |v| of each dim, however small the weights are beside the largest."""
import math

import pytest
import torch

from test_kv8_gpu import BF16, F32, build, compare, gpu_cache

pytestmark = pytest.mark.gpu


def attend(rows, heads, kv_heads, dim, dtype, change, window=0, sinks=0):
    K, V, table, q, kv_len, starts = build(rows, heads, kv_heads, dim, 64, 16, 17, dtype)
    change(K, V, table, q)
    cache = gpu_cache(K, V, table)
    out = cache.attend(q.cuda(), kv_len.cuda(), starts.cuda(), max_new=max(n for _, n in rows), window=window, sinks=sinks)
    cache.check()
    compare(out, rows, K, V, table, q, window, sinks, dtype)


SHAPES = [([(2500, 1), (700, 1)], 64), ([(900, 3)], 128), ([(70, 40)], 64), ([(1500, 60), (300, 60)], 128), ([(900, 300)], 64)]
IDS = ["tokens", "draft", "chunk", "chunks", "prompt"]


def dominant(at, gap, zero=True):
    """Position `at` of each row scores `gap` nats above 0 for every query, the rest of its block 0; its V is zero."""
    def change(K, V, table, q):
        q[..., 0] = 8.0
        for r in range(table.shape[0]):
            page, off = table[r, at // 64].long(), at % 64
            first = off // 16 * 16
            K.x[page, :, first:first + 16] = 0.0
            K.e[page, :, off // 16] = -2
            # 8 * x * 2^-2 / sqrt(dim) = gap
            K.x[page, :, off, 0] = float(torch.tensor(gap * math.sqrt(q.shape[2]) / 2).to(torch.float8_e4m3fn))
            if zero:
                V.x[page, :, off] = 0.0
    return change


@pytest.mark.parametrize("gap", [10, 14, 18, 22, 40, 60])
@pytest.mark.parametrize("rows,dim", SHAPES, ids=IDS)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_dominant_first_position_without_values(gap, rows, dim, dtype):
    """What the others contribute is all there is: weights of e^-gap and below."""
    attend(rows, 4, 2, dim, dtype, dominant(0, gap))


@pytest.mark.parametrize("gap", [18, 40])
@pytest.mark.parametrize("at", [17, 29])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_dominant_position_among_the_others(gap, at, dtype):
    """The dominant position is neither the first of its row nor of its tile; with a window that leaves it as a sink."""
    attend([(900, 1), (800, 1)], 8, 2, 64, dtype, dominant(at, gap))
    attend([(900, 50)], 8, 2, 64, dtype, dominant(at, gap))
    attend([(900, 50)], 8, 2, 64, dtype, dominant(at, gap), window=400, sinks=30)
    attend([(900, 2)], 8, 2, 64, dtype, dominant(at, gap, zero=False), window=300, sinks=30)


@pytest.mark.parametrize("spread", [11, 17, 24, 40, 90])
@pytest.mark.parametrize("rows,dim", SHAPES, ids=IDS)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_outlier_channels(spread, rows, dim, dtype):
    """Blocks of a V scale 2^spread above the others', whose tokens are zero in all dims but one."""
    def change(K, V, table, q):
        V.e[:] = -30
        for b in (0, 2):   # of each page: two of its four blocks
            V.e[:, :, b] = -30 + spread
            here = V.x[:, :, 16 * b:16 * b + 16]
            seen = ~torch.isnan(here)
            seen[..., 5] = False
            here[seen] = 0.0
    attend(rows, 4, 2, dim, dtype, change)


@pytest.mark.parametrize("spread", [17, 40, 90, 200])
@pytest.mark.parametrize("rows,dim", SHAPES, ids=IDS)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_outlier_channels_in_every_fifth_block(spread, rows, dim, dtype):
    """As above, in an order that gives each warp of a kernel blocks of both kinds."""
    def change(K, V, table, q):
        K.e.clamp_(max=-6)
        V.e[:] = -(spread // 2)
        for r in range(table.shape[0]):
            for b in range(0, 4 * table.shape[1], 5):
                page = table[r, b // 4].long()
                V.e[page, :, b % 4] += spread
                here = V.x[page, :, 16 * (b % 4):16 * (b % 4) + 16]
                seen = ~torch.isnan(here)
                seen[..., 5] = False
                here[seen] = 0.0
    attend(rows, 4, 2, dim, dtype, change)


@pytest.mark.parametrize("e", [-100, 100])
@pytest.mark.parametrize("rows,dim", SHAPES, ids=IDS)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scales_at_the_ends_of_their_range(e, rows, dim, dtype):
    """Scale bytes 27 and 227 in V, and in K with queries that bring the scores back."""
    K, V, table, q, kv_len, starts = build(rows, 4, 2, dim, 64, 16, 23, dtype)
    V.e[:] = e
    K.e[:] = e
    q = (q * 2.0 ** (-6 - e)).to(dtype)
    cache = gpu_cache(K, V, table)
    out = cache.attend(q.cuda(), kv_len.cuda(), starts.cuda(), max_new=max(n for _, n in rows))
    cache.check()
    V.e[:] = 0
    compare(out.double() * 2.0 ** -e, rows, K, V, table, q, 0, 0, dtype)


@pytest.mark.parametrize("new", [1, 2, 40])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_every_byte_of_v(new, dtype):
    """A token that sees one position gets its V: all finite e4m3 values, zeros and subnormals among them."""
    from graph_replay_gb300 import KV8Cache
    length = 256
    values = torch.arange(256, dtype=torch.uint8)
    values[0x7F], values[0xFF] = 0x7E, 0xFE
    v = values[(torch.arange(length)[:, None] * 7 + torch.arange(64)[None] * 5) % 256].view(1, 1, length, 64).contiguous()
    scale = torch.full((1, 1, length // 16), 127, dtype=torch.uint8)
    cache = KV8Cache(torch.zeros_like(v).cuda(), v.cuda(), scale.cuda(), scale.clone().cuda(), rows=1)
    for last in range(new, length + 1, new):
        out = cache.attend(torch.ones(new, 4, 64, dtype=dtype, device="cuda"), torch.tensor([last], dtype=torch.int32, device="cuda"),
                           torch.tensor([0, new], dtype=torch.int32, device="cuda"), max_new=new, window=1)
        want = v[0, 0, last - new:last].view(torch.float8_e4m3fn).double()[:, None].expand(new, 4, 64)
        # the weight and the sum are one number; its inverse and the products are rounded: four half steps of fp32.  A value
        # has 4 significant bits, so bf16 gives it back
        off = (out.double().cpu() - want).abs()
        assert bool((off <= want.abs() * (4 * 2.0 ** -24 if dtype == F32 else 0.0)).all()), last
    cache.check()


@pytest.mark.parametrize("byte", [1, 26, 228, 254])
@pytest.mark.parametrize("which", ["k_scale", "v_scale"])
@pytest.mark.parametrize("new", [1, 40])
def test_scales_out_of_range(byte, which, new):
    """They are flagged where a token reads their block, and other rows keep their results."""
    from graph_replay_gb300 import _binding as B
    rows = [(300, new), (300, new), (200, new)]
    K, V, table, q, kv_len, starts = build(rows, 4, 2, 64, 64, 16, 29, F32)
    cache = gpu_cache(K, V, table)
    args = dict(q_start=starts.cuda(), max_new=new, window=100, sinks=3)
    good = cache.attend(q.cuda(), kv_len.cuda(), **args)
    for block, seen in ((6, False), (0, True), (17, True)):   # blocks of row 1: between the sinks and the window, and in them
        scale = getattr(cache, which)
        at = (table[1, block // 4].long(), 1, block % 4)
        was = int(scale[at])
        scale[at] = byte
        out = cache.attend(q.cuda(), kv_len.cuda(), **args)
        if seen:
            with pytest.raises(B.DecError, match="0x20"):
                cache.check()
        else:
            cache.check()
            assert torch.equal(out, good)
        assert torch.equal(out[:new], good[:new]) and torch.equal(out[2 * new:], good[2 * new:])
        scale[at] = was
    assert torch.equal(cache.attend(q.cuda(), kv_len.cuda(), **args), good)
    cache.check()


# fp32 q over 32k positions: the error's norm over the result's.  Scores: the tensor core cuts each of its 8 (dim 128) or 4
# sums off at half a step of 2^-23 on the average, relative to scores of some 4 bits: 4 * 8 * 2^-24 = 2e-6 at the largest
# scores, half of it at the usual ones.  Exponential: 2^-22, its argument (up to 32) 2^-20 at the worst, a third on the
# average: 4e-7 each.  P V: 3 parts x 4 sums x 6 tiles are cut off before a fold, half a step of 2^-23 each of a sum that
# is half grown on the average: 72 * 2^-24 / 2 / 2 (a step is between 2^-24 and 2^-23 of the sum) = 1.1e-6.  Together
# 1.6e-6 as independent errors, 3e-6 with a factor for what is not.  Without the folds it is 7e-6, with weights of one
# part 1e-4
@pytest.mark.parametrize("new,heads,kv_heads,dim", [(1, 4, 2, 128), (1, 8, 2, 64), (64, 4, 2, 64), (64, 4, 1, 128)])
def test_fp32_error_over_long_contexts(new, heads, kv_heads, dim):
    import _kv8 as R
    rows = [(32767, new)]
    K, V, table, q, kv_len, starts = build(rows, heads, kv_heads, dim, 64, 64, 41, F32, poison=False)
    K.e[:], V.e[:] = -6, -6          # values of about 1, scores of about 1
    cache = gpu_cache(K, V, table)
    out = cache.attend(q.cuda(), kv_len.cuda(), starts.cuda(), max_new=new).double().cpu()
    cache.check()
    at = table[0].long()
    want, _, _ = R.attend(q.double(), K.values(at), V.values(at), torch.arange(32767 - new, 32767))
    assert float((out - want).norm() / want.norm()) <= 3e-6


def test_nan_behind_a_thousand_tiles():
    """CTAs of more than 1024 tiles of 64 positions, where the marks of tiles that hold a NaN come round again."""
    from graph_replay_gb300 import KV8Cache
    heads, length, new, window = 160, 64 * 1100, 60, 70000     # enough heads that no CTA shares its positions with another
    cache = KV8Cache.empty(1, length, heads, 64, scale_block=64)
    cache.v.fill_(0x38)                                         # 1.0 everywhere; K is zero, so every result is 1
    first = length - new
    early, late = first + 30 - window, 1029 * 64 + 5   # tile of `early` and tile 1029, whose marks are one
    assert (early // 64) % 1024 == 1029 % 1024 and 0 <= early and late // 64 == 1029
    cache.v[0, 0, early, 3] = 0x7F
    cache.v[0, 1, late, 7] = 0xFF
    cache.v[0, 2, first - window - 64, 9] = 0x7F                # nobody sees it
    out = cache.attend(torch.ones(new, heads, 64, device="cuda", dtype=BF16), torch.tensor([length], dtype=torch.int32, device="cuda"),
                       torch.tensor([0, new], dtype=torch.int32, device="cuda"), max_new=new, window=window)
    cache.check()
    nan = torch.zeros(new, heads, 64, dtype=torch.bool, device="cuda")
    nan[:30, 0, 3] = True            # token t sees positions from first + t - window + 1 on: t < 30 see `early`
    nan[:, 1, 7] = True
    assert torch.equal(torch.isnan(out), nan) and bool((out[~nan] == 1).all())


@pytest.mark.parametrize("power", [10, 20, 24, 25, 27, 30, 40, 60])
@pytest.mark.parametrize("rows,dim", SHAPES, ids=IDS)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_one_score_far_above(power, rows, dim, dtype):
    """Position 5 scores 1.25 * 2^power / sqrt(dim), the others 0: the results are its V, also where scores lie further
    apart than 1 in fp32."""
    K, V, table, q, kv_len, starts = build(rows, 4, 2, dim, 64, 16, 17, dtype)
    q = torch.zeros_like(q)
    q[..., 0] = 1.0
    K.x.zero_()
    K.e.zero_()
    K.x[table[:, 0].long(), :, 5, 0] = 1.25
    K.e[table[:, 0].long(), :, 0] = power
    cache = gpu_cache(K, V, table)
    out = cache.attend(q.cuda(), kv_len.cuda(), starts.cuda(), max_new=max(n for _, n in rows))
    cache.check()
    for r, (l, n) in enumerate(rows):
        v = V.values(table[r].long())[:, 5].repeat_interleave(2, 0)
        off = (out[starts[r]:starts[r + 1]].double().cpu() - v)[max(5 - (l - n), 0):].abs()
        # the weight and the sum are one number; its inverse and the products are rounded: four half steps of fp32, then the
        # result's own (a value of 4 bits, so bf16 has it)
        assert bool((off <= v.abs() * 4 * 2.0 ** -24).all() if dtype == F32 else (off == 0).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_steps_that_wait_in_long_pieces(dtype):
    """640 heads of 131072 positions: a warp has more steps than it has marks.  One position of each head, at other places,
    scores 30 nats above the others and holds no V; the 15 others of its step are a ten-thousandth of the result."""
    from graph_replay_gb300 import KV8Cache
    heads, length = 640, 1 << 17
    cache = KV8Cache.empty(1, length, heads, 64)
    cache.v.fill_(0x38)                                    # 1.0
    h = torch.arange(heads, device="cuda")
    at = (h * 7919 + 5) * 131 % length
    cache.k[0, h, at, 0] = int(torch.tensor(120.0).to(torch.float8_e4m3fn).view(torch.uint8))
    cache.k_scale[0, h, at // 64] = 125                    # 120 / 4
    cache.v[0, h, at] = 0
    q = torch.zeros(1, heads, 64, dtype=dtype, device="cuda")
    q[..., 0] = 8.0                                        # 8 * 30 / sqrt(64)
    out = cache.attend(q, torch.tensor([length], dtype=torch.int32, device="cuda"))
    cache.check()
    w = (length - 1) * math.exp(-30.0)
    want = w / (1 + w)
    # the exponential and its argument of 43 in fp32 (2^-21 + 43 * 2^-24), the sums (131072 equal terms, each rounding at
    # most half a step of the sum: sqrt(n) * 2^-24), the type's half step; with fp32 a fifth of what the 15 weigh
    tol = want * (2.0 ** -21 + 43 * 2.0 ** -24 + math.sqrt(length) * 2.0 ** -24 + torch.finfo(dtype).eps / 2)
    assert float((out.double() - want).abs().max()) <= tol
