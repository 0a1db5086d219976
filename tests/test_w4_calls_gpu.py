"""The 4-bit weights' calls as programs make them: recorded, on several streams and threads, on views, in place, with values
that are not finite, and together with the 8-bit K/V cache as one layer."""
import threading

import pytest
import torch

import _w4 as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def W():
    from graph_replay_gb300 import W4Weight, build
    build.build()
    return W4Weight


def normal(*shape, seed=0, dtype=torch.float32):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


SIZES = [(1, 512, 1152, 64, torch.float32), (8, 300, 4096, 128, torch.bfloat16), (8, 512, 14336, 128, torch.float32),
         (40, 640, 2048, 32, torch.bfloat16), (200, 384, 1152, 64, torch.float32)]


@pytest.mark.parametrize("m, n, k, group, dt", SIZES)
def test_recorded_calls_follow_their_inputs(W, m, n, k, group, dt):
    a, b = W(*R.random_matrix(n, k, group, 1)), W(*R.random_matrix(n, k, group, 2))
    x, h, gain = normal(m, k, seed=1, dtype=dt), normal(m, n, seed=2, dtype=dt), normal(k, seed=3, dtype=dt)
    y, z = torch.empty_like(h), torch.empty_like(h)
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        a.linear(x, residual=h, norm=gain, out=y)
        a.glu(b, x, out=z)
        a.linear(x, residual=y, out=y)         # in place, behind the first
    for seed in (5, 6):
        x.copy_(normal(m, k, seed=seed, dtype=dt))
        h.copy_(normal(m, n, seed=seed + 9, dtype=dt))
        graph.replay()
        want = a.linear(x, residual=h, norm=gain)
        assert torch.equal(z, a.glu(b, x))
        assert torch.equal(y, a.linear(x, residual=want))
    a.check()


def test_streams_and_threads(W):
    """Calls of one weight on several streams from several threads: each gives what it gives alone."""
    cases = [(W(*R.random_matrix(n, k, g, i)), normal(m, k, seed=i, dtype=dt)) for i, (m, n, k, g, dt) in enumerate(SIZES)]
    want = [w.linear(x) for w, x in cases]
    torch.cuda.synchronize()
    bad = []

    def work(t):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for i in range(25):
                w, x = cases[(i + t) % len(cases)]
                y = w.linear(x)
                s.synchronize()
                if not torch.equal(y, want[(i + t) % len(cases)]):
                    bad.append((t, i))
    threads = [threading.Thread(target=work, args=(t,)) for t in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    cases[0][0].check()


@pytest.mark.parametrize("m", [1, 5, 30])
def test_views_and_types(W, m):
    """x and out as parts of wider matrices, fp32 results of bf16 activations, a gain of the other type; what lies beside is kept."""
    n, k = 130, 384
    c, s = R.random_matrix(n, k, 64, 3)
    w = W(c, s)
    wide = normal(m, 3 * k, seed=1, dtype=torch.bfloat16)
    x = wide[:, k:2 * k]
    out = torch.full((m, n + 7), 9.0, device="cuda")
    gain = 1.0 + 0.1 * normal(k, seed=4)
    w.linear(x, norm=gain, out=out[:, 3:3 + n])
    a = R.activation(x, gain, 1e-5)
    want = a @ R.values(c, s).T
    R.close(out[:, 3:3 + n], want, R.product_bound(a, R.values(c, s), 21 if m <= 8 else 11, k) + 2.0 ** -21 * want.abs())
    assert (out[:, :3] == 9.0).all() and (out[:, 3 + n:] == 9.0).all()
    y = w.linear(x, dtype=torch.float32)
    R.close(y, x.double() @ R.values(c, s).T, R.product_bound(x.double(), R.values(c, s), 40, k))


def test_nothing_and_one(W):
    w = W(*R.random_matrix(64, 128, 128, 1))
    for dt in (torch.float32, torch.bfloat16):
        assert w.linear(torch.empty(0, 128, device="cuda", dtype=dt)).shape == (0, 64)
        assert w.glu(w, torch.empty(0, 128, device="cuda", dtype=dt)).shape == (0, 64)
    assert torch.equal(w.linear(torch.zeros(3, 128, device="cuda"), norm=torch.ones(128, device="cuda")), torch.zeros(3, 64, device="cuda"))


@pytest.mark.parametrize("m", [3, 40])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_values_that_are_not_finite(W, m, dt):
    """A NaN or an infinity stays in its token; a NaN scale in its output row."""
    n, k = 96, 256
    c, s = R.random_matrix(n, k, 64, 5)
    s = s.clone()
    s[7, 2] = float("nan")
    w = W(c, s)
    x = normal(m, k, seed=2, dtype=dt)
    x[1, 5] = float("nan")
    x[2, 100] = float("inf")
    y = w.linear(x)
    g = w.glu(w, x)
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[7] = False
    for out in (y, g):
        assert torch.isnan(out[:, 7]).all() and torch.isnan(out[1]).all()
        assert torch.isfinite(out[0][keep]).all() and torch.isfinite(out[3:][:, keep]).all()
    assert not torch.isfinite(y[2]).any()
    clean = x.clone()
    clean[1:3] = 0
    assert torch.equal(w.linear(clean)[0][keep], y[0][keep])


@pytest.mark.parametrize("m", [2, 20])
def test_far_sizes(W, m):
    """Large and small values: results within fp32 come out, in tokens and rows of unlike size."""
    n, k = 64, 256
    c, s = R.random_matrix(n, k, 128, 5, spread=0.0)
    row = torch.exp2(torch.linspace(-60, 60, n, device="cuda"))[:, None]
    w = W(c, (s.float() * row).bfloat16())
    x = normal(m, k, seed=1) * torch.exp2(torch.linspace(-50, 50, m, device="cuda"))[:, None]
    v = R.values(c, w.scales)
    want = x.double() @ v.T
    got = w.linear(x)
    R.close(got, want, R.product_bound(x.double(), v, 21, k))


@pytest.mark.parametrize("m", [4, 24])
def test_scales_of_one_row_far_apart(W, m):
    """Groups 2^20 apart in one row, fp32 tokens that meet only the small ones."""
    n, k = 64, 512
    c, s = R.random_matrix(n, k, 128, 6)
    s = s * torch.tensor([1.0, 2.0 ** -20, 1.0, 2.0 ** -20], device="cuda", dtype=torch.bfloat16)
    w = W(c, s)
    x = normal(m, k, seed=2)
    x[1, :128] = x[1, 256:384] = 0.0
    v = R.values(c, s)
    want = x.double() @ v.T
    R.close(w.linear(x), want, R.product_bound(x.double(), v, 21, k))


def test_one_layer_of_a_program_with_its_own_cache(W):
    """RMSNorm and QKV, RoPE by the caller, the 8-bit cache, output projection, gated block: a prompt, then single tokens."""
    from graph_replay_gb300 import KV8Cache
    d, heads, kv, hd, f, rows = 512, 8, 2, 64, 1024, 3
    wq, wo, wg, wu, wd = (W.quantize(normal(a, b, seed=i) * 0.03, 64) for i, (a, b) in
                          enumerate([((heads + 2 * kv) * hd, d), (d, heads * hd), (f, d), (f, d), (d, f)]))
    g1, g2 = 1 + 0.1 * normal(d, seed=7), 1 + 0.1 * normal(d, seed=8)
    cache = KV8Cache.empty(rows, 128, kv, hd)

    def layer(x, kv_len, q_start, max_new, c):
        qkv = wq.linear(x, norm=g1).view(x.shape[0], heads + 2 * kv, hd)
        q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
        c.append(k, v, kv_len, q_start=q_start, max_new=max_new)
        o = c.attend(q, kv_len, q_start=q_start, max_new=max_new).reshape(x.shape[0], heads * hd)
        x = wo.linear(o, residual=x)
        return wd.linear(wg.glu(wu, x, norm=g2), residual=x, out=x)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    x = normal(17 + 5 + 30, d, seed=11)
    prompt = layer(x, i32(17, 5, 30), i32(0, 17, 22, 52), 30, cache)
    step = layer(normal(rows, d, seed=12), i32(18, 6, 31), None, 1, cache)

    # the same in fp64 over the values that were stored
    val = {w: R.values(w.codes, w.scales) for w in (wq, wo, wg, wu, wd)}

    def stored(c, which, r):
        b = getattr(c, which)[r].view(torch.float8_e4m3fn).double()
        e = torch.exp2(getattr(c, which + "_scale")[r].double() - 127.0).repeat_interleave(c.scale_block, 1)
        return b * e[..., None]

    def plain(x, r, n, upto):
        x = x.double()
        q = (R.activation(x, g1, 1e-5) @ val[wq].T).view(-1, heads + 2 * kv, hd)[:, :heads]
        out = torch.empty(x.shape[0], heads, hd, dtype=torch.float64, device="cuda")
        for t in range(x.shape[0]):
            p = upto - n + t + 1
            for a in range(heads):
                kk, vv = stored(cache, "k", r)[a // 4, :p], stored(cache, "v", r)[a // 4, :p]
                out[t, a] = torch.softmax(q[t, a] @ kk.T / 8.0, -1) @ vv
        x = x + out.view(x.shape[0], -1) @ val[wo].T
        h = R.activation(x, g2, 1e-5)
        return x + R.glu("silu", h @ val[wg].T, h @ val[wu].T) @ val[wd].T
    # (a block's scale may have grown with the last token: compare the steps, whose cache is the final one)
    x1 = normal(rows, d, seed=12)
    for r, l in enumerate((18, 6, 31)):
        want = plain(x1[r:r + 1], r, 1, l)[0]
        assert (step[r].double() - want).norm() <= 1e-5 * want.norm()
    assert torch.isfinite(prompt).all()
    wq.check()
    cache.check()


@pytest.mark.parametrize("m, n, k, dt", [(8, 40, 32768, torch.float32), (8, 3000, 28672, torch.float32), (16, 100, 65536, torch.bfloat16),
                                         (1, 9, 1 << 19, torch.float32), (2, 16, 1 << 20, torch.bfloat16)])
def test_many_columns(W, m, n, k, dt):
    """More than the activations' shared memory holds at once."""
    c, s = R.random_matrix(n, k, 128, 5)
    x = normal(m, k, seed=1, dtype=dt)
    w, v = W(c, s), R.values(c, s)
    R.close(w.linear(x), x.double() @ v.T, R.product_bound(x.double(), v, 21 if dt == torch.float32 else 40, k))
    w.check()


def test_out_beside_x_and_over_it(W):
    from graph_replay_gb300 import _binding as B
    w = W(*R.random_matrix(128, 128, 128, 5))
    wide = normal(6, 512, seed=1)
    x = wide[:, :128].clone()
    want = w.linear(x)
    assert torch.equal(w.linear(wide[:, :128], out=wide[:, 128:256]), want)
    assert torch.equal(wide[:, :128], x)
    for out in (wide[:, :128], wide[:, 64:192], wide[1:].view(-1)[:6 * 128].view(6, 128)[:6]):
        with pytest.raises(B.DecError, match="overlaps"):
            w.linear(wide[:, :128], out=out)
