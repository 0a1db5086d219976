"""The 8-bit K/V cache on the GPU against its definitions in 64 bits: appending, attention for single tokens and
prompts, masks, lengths, layouts, streams and graphs."""
import math

import pytest
import torch

import _kv8 as R

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def gpu_cache(K, V, table):
    from graph_replay_gb300 import KV8Cache
    (kb, ks), (vb, vs) = K.bytes(), V.bytes()
    return KV8Cache(kb.cuda(), vb.cuda(), ks.cuda(), vs.cuda(), page_table=table.cuda())


def starts_of(ns):
    s = [0]
    for n in ns:
        s.append(s[-1] + n)
    return torch.tensor(s, dtype=torch.int32)


def build(rows, heads, kv_heads, dim, page, block, seed, dtype, poison=True):
    """rows: [(length, new tokens)].  Positions behind a row's end hold NaN."""
    g = torch.Generator().manual_seed(seed)
    per = max(1, -(-max(l for l, _ in rows) // page)) + 1
    table = R.table_of(len(rows), per, g)
    K, V = (R.random_store(len(rows) * per + 3, kv_heads, page, dim, block, g) for _ in range(2))
    for r, (l, _) in enumerate(rows):
        if not poison:
            break
        for s in (K, V):
            for j in range(l, per * page):
                s.x[table[r, j // page].long(), :, j % page] = math.nan
    total = sum(n for _, n in rows)
    q = torch.randn(total, heads, dim, generator=g).to(dtype)
    kv_len = torch.tensor([l for l, _ in rows], dtype=torch.int32)
    return K, V, table, q, kv_len, starts_of([n for _, n in rows])


def compare(out, rows, K, V, table, q, window, sinks, dtype, scale=None):
    t = 0
    for r, (l, n) in enumerate(rows):
        p = torch.arange(l - n, l)
        o, mass, score = R.attend(q[t:t + n].double(), K.values(table[r].long()), V.values(table[r].long()), p, window, sinks, scale)
        got = out[t:t + n].double().cpu()
        assert bool((torch.isnan(got) == torch.isnan(o)).all()), f"row {r}: NaN in other places"
        off = torch.where(torch.isnan(o), torch.zeros_like(o), (got - o).abs())
        lim = R.bound(mass.nan_to_num(0.0), score, o.nan_to_num(0.0), dtype, q.shape[2], max(l, 1))
        worst = float((off / lim).max()) if off.numel() else 0.0
        assert worst <= 1.0, f"row {r} (length {l}, {n} new): {worst:.3g} of what the arithmetic allows"
        t += n


TOKEN_ROWS = [
    [(1, 1)], [(15, 1)], [(16, 1)], [(17, 1)], [(63, 1)], [(64, 1)], [(65, 1)], [(129, 1)], [(2500, 1)],
    [(0, 1), (1, 1), (700, 1), (0, 1), (64, 1), (333, 1)],
    [(33, 1)] * 40,
]


@pytest.mark.parametrize("rows", TOKEN_ROWS, ids=lambda r: "-".join(str(l) for l, _ in r[:6]))
@pytest.mark.parametrize("heads,kv_heads,dim,dtype", [(8, 2, 128, F32), (8, 2, 128, BF16), (4, 4, 64, F32), (16, 2, 64, BF16),
                                                      (16, 1, 128, F32), (10, 2, 64, F32), (3, 1, 128, BF16)])
def test_token_attention(rows, heads, kv_heads, dim, dtype):
    page, block = (16, 16) if kv_heads == 2 else (128, 64)
    K, V, table, q, kv_len, _ = build(rows, heads, kv_heads, dim, page, block, 7, dtype)
    cache = gpu_cache(K, V, table)
    out = cache.attend(q.cuda(), kv_len.cuda())
    cache.check()
    compare(out, rows, K, V, table, q, 0, 0, dtype)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 4), (64, 0), (64, 33), (100, 200), (1000, 4), (5000, 3)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_token_window(window, sinks, dtype):
    rows = [(1, 1), (8, 1), (65, 1), (900, 1), (0, 1), (1111, 1)]
    K, V, table, q, kv_len, _ = build(rows, 8, 2, 64, 32, 16, 3, dtype)
    cache = gpu_cache(K, V, table)
    out = cache.attend(q.cuda(), kv_len.cuda(), window=window, sinks=sinks)
    cache.check()
    compare(out, rows, K, V, table, q, window, sinks, dtype)


PROMPTS = [
    # rows, heads, kv_heads, dim, page, block, window, sinks
    ([(2, 2)], 4, 2, 128, 16, 16, 0, 0),
    ([(5, 3), (9, 4), (0, 0), (4, 1)], 8, 2, 64, 16, 16, 0, 0),          # up to 16 query rows of a K/V head
    ([(300, 2), (7, 2)], 16, 2, 128, 64, 64, 0, 0),
    ([(300, 4), (7, 3), (40, 4)], 4, 1, 64, 32, 32, 5, 2),
    ([(33, 33)], 8, 2, 128, 64, 64, 0, 0),
    ([(128, 128), (1, 1), (129, 129)], 4, 4, 64, 16, 16, 0, 0),
    ([(700, 257), (3, 3), (0, 0), (513, 1)], 8, 2, 128, 128, 128, 0, 0),
    ([(1500, 40), (64, 64)], 12, 4, 64, 64, 32, 0, 0),                   # groups of 3
    ([(400, 300)], 40, 1, 128, 16, 16, 0, 0),                            # groups of 40
    ([(600, 600), (77, 50)], 8, 2, 64, 32, 32, 1, 0),
    ([(600, 600), (77, 50)], 8, 2, 128, 32, 32, 1, 1),
    ([(1000, 500), (130, 130)], 8, 2, 128, 64, 16, 100, 4),
    ([(1000, 500), (130, 130)], 4, 2, 64, 64, 64, 64, 200),
    ([(5, 9), (2, 40)], 8, 2, 64, 16, 16, 0, 0),                         # more tokens than positions: the first see nothing
    ([(4000, 70)], 4, 1, 128, 64, 64, 0, 0),                             # few rows, many positions
    ([(4000, 70), (90, 90)], 4, 1, 64, 64, 64, 900, 130),
]


@pytest.mark.parametrize("case", PROMPTS, ids=lambda c: f"{c[0][0][0]}x{c[0][0][1]}-h{c[1]}-{c[2]}-d{c[3]}-w{c[6]}-s{c[7]}")
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prompt_attention(case, dtype):
    rows, heads, kv_heads, dim, page, block, window, sinks = case
    K, V, table, q, kv_len, starts = build(rows, heads, kv_heads, dim, page, block, 11, dtype)
    cache = gpu_cache(K, V, table)
    out = cache.attend(q.cuda(), kv_len.cuda(), q_start=starts.cuda(), max_new=max(n for _, n in rows), window=window, sinks=sinks)
    cache.check()
    compare(out, rows, K, V, table, q, window, sinks, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("new", [1, 3, 60])
def test_large_scores_and_scales(dtype, new):
    # peaked softmax, K and V exponents far apart between blocks, a scale of the caller's own
    g = torch.Generator().manual_seed(1)
    rows = [(400, new)]
    K, V, table, q, kv_len, starts = build(rows, 4, 2, 64, 64, 16, 5, dtype)
    K.e = torch.randint(-12, 2, K.e.shape, generator=g)
    V.e = torch.randint(-40, 14, V.e.shape, generator=g)
    cache = gpu_cache(K, V, table)
    out = cache.attend(q.cuda(), kv_len.cuda(), q_start=starts.cuda(), max_new=new, scale=0.05)
    compare(out, rows, K, V, table, q, 0, 0, dtype, scale=0.05)


@pytest.mark.parametrize("new", [1, 3, 60])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_nan_stays_where_it_is_seen(new, dtype):
    """NaN in V (one dim) and K at positions that only some tokens see: those tokens', and no other's, results."""
    rows = [(300, new)]
    window, sinks = 40, 3
    K, V, table, q, kv_len, starts = build(rows, 4, 2, 64, 16, 16, 9, dtype)
    def put(s, j, h, d):
        s.x[table[0, j // 16].long(), h, j % 16, d] = math.nan
    put(V, 299, 0, 5)                  # the last token alone sees it
    put(V, 299 - new // 2, 1, 7)       # half of the tokens see it
    put(V, 300 - new - window, 0, 9)   # just behind the first token's window
    put(V, 100, 1, slice(None))        # nobody's
    put(K, 120, 0, 1)
    put(K, 299, 1, 63)
    cache = gpu_cache(K, V, table)
    out = cache.attend(q.cuda(), kv_len.cuda(), q_start=starts.cuda(), max_new=new, window=window, sinks=sinks)
    compare(out, rows, K, V, table, q, window, sinks, dtype)


@pytest.mark.parametrize("new", [1, 40])
def test_strided_tokens_and_rows_behind_the_last(new):
    rows = [(50, new), (77, new)]
    K, V, table, q, kv_len, starts = build(rows, 8, 2, 64, 16, 16, 2, BF16)
    cache = gpu_cache(K, V, table)
    total = q.shape[0]
    packed = torch.full((total + 5, 12, 64), math.nan, dtype=BF16, device="cuda")   # q beside k and v heads
    packed[:total, :8] = q.cuda()
    wide = torch.full((total + 5, 10, 64), 7.0, dtype=BF16, device="cuda")
    out = cache.attend(packed[:, :8], kv_len.cuda(), q_start=starts.cuda(), max_new=new, out=wide[:, 1:9])
    cache.check()
    compare(out, rows, K, V, table, q, 0, 0, BF16)
    assert bool((wide[total:] == 7).all()) and bool((wide[:, 0] == 7).all()) and bool((wide[:, 9] == 7).all())


@pytest.mark.parametrize("new", [1, 40])
def test_entries_out_of_range(new):
    from graph_replay_gb300 import _binding as B
    rows = [(50, new), (77, new), (60, new), (64, new)]
    K, V, table, q, kv_len, starts = build(rows, 4, 2, 64, 16, 16, 2, F32)
    good = gpu_cache(K, V, table).attend(q.cuda(), kv_len.cuda(), q_start=starts.cuda(), max_new=new)
    cap = table.shape[1] * 16
    for bad in (cap + 1, -1, 2 ** 31 - 1):
        cache = gpu_cache(K, V, table)
        lens = kv_len.clone()
        lens[1] = bad
        out = torch.full_like(good, 3.0)
        cache.attend(q.cuda(), lens.cuda(), q_start=starts.cuda(), max_new=new, out=out)
        with pytest.raises(B.DecError) as e:
            cache.check()
        assert e.value.status == B.DEC_E_DEVICE_FAULT and "0x2" in str(e.value)
        cache.check()   # cleared
        assert bool((out[new:2 * new] == 3).all()) and torch.equal(out[:new], good[:new]) and torch.equal(out[2 * new:], good[2 * new:])
    # a page that is needed and is none: the others' rows keep their results
    tb = table.clone()
    tb[2, 1], tb[0, -1] = 10 ** 6, -5      # row 0's last page is behind its end: not needed
    cache = gpu_cache(K, V, tb)
    out = cache.attend(q.cuda(), kv_len.cuda(), q_start=starts.cuda(), max_new=new)
    with pytest.raises(B.DecError, match="0x8"):
        cache.check()
    for r in (0, 1, 3):
        assert torch.equal(out[r * new:(r + 1) * new], good[r * new:(r + 1) * new])
    # token ranges: descending, behind the end, longer than max_new
    for change in ((1, 3 * new + 1), (4, 4 * new + 9)):
        s = starts.clone()
        s[change[0]] = change[1]
        cache = gpu_cache(K, V, table)
        cache.attend(q.cuda(), kv_len.cuda(), q_start=s.cuda(), max_new=new)
        with pytest.raises(B.DecError, match="0x2"):
            cache.check()


# ---- append ----

def append_case(rows, kv_heads, dim, page, block, dtype, seed=4, grow=4.0, stride=0):
    g = torch.Generator().manual_seed(seed)
    per = max(1, -(-max(l for l, _ in rows) // page))
    table = R.table_of(len(rows), per, g)
    K, V = (R.random_store(len(rows) * per + 3, kv_heads, page, dim, block, g, spread=2) for _ in range(2))
    total = sum(n for _, n in rows)
    k = (torch.randn(total, kv_heads, dim, generator=g) * torch.exp2(torch.randint(-3, 5, (total, 1, 1), generator=g).float()) * grow).to(dtype)
    v = torch.randn(total, kv_heads, dim, generator=g).to(dtype)
    return K, V, table, k, v


def same_bytes(cache, K, V):
    for got, sc, s in ((cache.k, cache.k_scale, K), (cache.v, cache.v_scale, V)):
        b, e = s.bytes()
        assert torch.equal(sc.cpu(), e)
        x, y = got.cpu().view(torch.float8_e4m3fn).float(), b.view(torch.float8_e4m3fn).float()
        assert bool(((x == y) | (torch.isnan(x) & torch.isnan(y))).all())


@pytest.mark.parametrize("rows", [[(1, 1)], [(17, 1), (0, 1), (16, 1), (40, 1)], [(300, 300)], [(77, 60), (5, 5), (9, 0), (3, 8)],
                                  [(130, 3), (128, 128)]], ids=str)
@pytest.mark.parametrize("kv_heads,dim,page,block", [(2, 128, 16, 16), (3, 64, 64, 32), (1, 128, 128, 128), (2, 64, 64, 64)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_append(rows, kv_heads, dim, page, block, dtype):
    K, V, table, k, v = append_case(rows, kv_heads, dim, page, block, dtype)
    cache = gpu_cache(K, V, table)
    starts = starts_of([n for _, n in rows])
    lens = torch.tensor([l for l, _ in rows], dtype=torch.int32)
    for _ in range(2):   # a second time changes nothing: the exponents have grown, the earlier bytes stay
        cache.append(k.cuda(), v.cuda(), lens.cuda(), q_start=starts.cuda(), max_new=max(n for _, n in rows))
        cache.check()
        for s, x in ((K, k), (V, v)):
            for r, (l, n) in enumerate(rows):
                s.append(table[r], l - n, x[starts[r]:starts[r + 1]].double())
        same_bytes(cache, K, V)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_append_extremes(dtype):
    rows = [(48, 48)]
    K, V, table, k, v = append_case(rows, 1, 64, 16, 16, dtype)
    k[:16] = 0.0
    k[16:32] = torch.tensor([448.0, 449.0, 2.0 ** -50, -3.0])[torch.arange(16) % 4][:, None, None].to(dtype)
    k[33], k[34], k[35] = math.nan, math.inf, -math.inf
    v[0], v[1], v[2] = 3e38, 448.0 * 2.0 ** 60, -1e-30
    v[16:32] = 1e-38
    cache = gpu_cache(K, V, table)
    cache.append(k.cuda(), v.cuda(), torch.tensor([48], dtype=torch.int32).cuda(), q_start=torch.tensor([0, 48], dtype=torch.int32).cuda(), max_new=48)
    K.append(table[0], 0, k.double())
    V.append(table[0], 0, v.double())
    same_bytes(cache, K, V)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("byte", [188, 240, 253, 255])
def test_append_to_a_block_of_larger_scale(byte, dtype):
    """A caller's own scale bytes go beyond those that append writes: the block keeps its exponent, infinities are NaN."""
    from graph_replay_gb300 import KV8Cache
    c = KV8Cache.empty(1, 64, 1, 64, scale_block=16)
    c.k_scale[:, :, 0] = byte
    c.v_scale[:, :, 0] = byte
    x = torch.zeros(2, 1, 64, dtype=dtype)
    x[0, 0, :6] = torch.tensor([math.inf, -math.inf, math.nan, 1.0, 2.0 ** (byte - 127 - 3), -3.0 * 2.0 ** (byte - 127 - 9)])
    c.append(x.cuda(), x.cuda(), torch.tensor([3], dtype=torch.int32, device="cuda"),
             torch.tensor([0, 2], dtype=torch.int32, device="cuda"), max_new=2)
    c.check()
    for pool, scale in ((c.k, c.k_scale), (c.v, c.v_scale)):
        assert int(scale[0, 0, 0]) == byte
        got = pool[0, 0, 1].view(torch.float8_e4m3fn).float().cpu()
        assert bool(got[:3].isnan().all())
        assert got[3:6].tolist() == [0.0, 2.0 ** -3, -3.0 * 2.0 ** -9] and not got[6:].any()


def test_append_from_a_packed_matrix_and_bad_entries():
    from graph_replay_gb300 import _binding as B
    rows = [(20, 3), (40, 2), (8, 8)]
    K, V, table, k, v = append_case(rows, 2, 64, 16, 16, BF16)
    starts, lens = starts_of([3, 2, 8]), torch.tensor([20, 40, 8], dtype=torch.int32)
    qkv = torch.zeros(13, 12, 64, dtype=BF16, device="cuda")
    qkv[:, 8:10], qkv[:, 10:] = k.cuda(), v.cuda()
    tb = table.clone()
    tb[1, 2] = -1                     # row 1's new tokens have no page
    lens[2] = tb.shape[1] * 16 + 1    # row 2 is out of range
    cache = gpu_cache(K, V, tb)
    cache.append(qkv[:, 8:10], qkv[:, 10:], lens.cuda(), q_start=starts.cuda(), max_new=8)
    with pytest.raises(B.DecError, match="0xa"):
        cache.check()
    K.append(table[0], 17, k[:3].double())
    V.append(table[0], 17, v[:3].double())
    same_bytes(cache, K, V)


# ---- together ----

@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 2)])
def test_prompt_then_tokens(window, sinks):
    """A prompt appended and attended, then token by token: each result as the definition says for what is stored by then."""
    from graph_replay_gb300 import KV8Cache
    g = torch.Generator().manual_seed(0)
    kv_heads, heads, dim, block = 2, 8, 64, 16
    cache = KV8Cache.empty(2, 64, kv_heads, dim, scale_block=block)
    K, V = (R.Store(2, kv_heads, 64, dim, block) for _ in range(2))
    at = [0, 0]
    for ns in ([37, 21], [1, 1], [1, 1], [3, 2], [1, 0], [12, 20], [1, 1]):
        total = sum(ns)
        q, k, v = (torch.randn(total, h, dim, generator=g) for h in (heads, kv_heads, kv_heads))
        starts = starts_of(ns)
        at = [a + n for a, n in zip(at, ns)]
        lens = torch.tensor(at, dtype=torch.int32).cuda()
        cache.append(k.cuda(), v.cuda(), lens, q_start=starts.cuda(), max_new=max(ns))
        out = cache.attend(q.cuda(), lens, q_start=starts.cuda(), max_new=max(ns), window=window, sinks=sinks)
        for r in range(2):
            a, b = int(starts[r]), int(starts[r + 1])
            K.append([r], at[r] - ns[r], k[a:b].double())
            V.append([r], at[r] - ns[r], v[a:b].double())
        compare(out, list(zip(at, ns)), K, V, torch.tensor([[0], [1]]), q, window, sinks, F32)
    same_bytes(cache, K, V)
    cache.check()


def test_graphs_and_streams():
    """One recorded step serves every length; two graphs and an eager call on other streams do not meet."""
    rows = [(900, 1), (33, 1), (2000, 1)]
    K, V, table, q, kv_len, _ = build(rows, 8, 2, 128, 64, 64, 21, F32, poison=False)
    cache = gpu_cache(K, V, table)
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    qs = [q.cuda(), torch.randn(q.shape, device="cuda"), torch.randn(q.shape, device="cuda")]
    news = [torch.randn(3, 2, 128, device="cuda") for _ in range(2)]
    want = [cache.attend(x, kv_len.cuda()).clone() for x in qs]
    outs = [torch.empty_like(qs[0]) for _ in range(2)]
    graphs, streams = [], [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for i in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=streams[i]):
            cache.attend(qs[i], lens, out=outs[i])
        graphs.append(gr)
    for _ in range(20):
        lens.copy_(kv_len)
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        with torch.cuda.stream(streams[2]):
            eager = cache.attend(qs[2], lens)
        torch.cuda.synchronize()
        for got, ref in zip(outs + [eager], want):
            assert torch.equal(got, ref)
    # the same graph at another length, with an append before it in a second recording
    lens.copy_(torch.tensor([100, 1, 1999], dtype=torch.int32))
    graphs[0].replay()
    torch.cuda.synchronize()
    compare(outs[0], [(100, 1), (1, 1), (1999, 1)], K, V, table, q, 0, 0, F32)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=streams[0]):
        cache.append(news[0], news[1], lens)
        cache.attend(qs[0], lens, out=outs[0])
    gr.replay()
    torch.cuda.synchronize()
    for s, x in ((K, news[0]), (V, news[1])):
        for r, l in enumerate((100, 1, 1999)):
            s.append(table[r], l - 1, x[r:r + 1].double().cpu())
    compare(outs[0], [(100, 1), (1, 1), (1999, 1)], K, V, table, q, 0, 0, F32)
    cache.check()


def test_threads_on_one_stream():
    """Calls of several threads on one stream share the cache's workspace; splits and their join stay together."""
    import threading
    rows = [(3000, 16)]
    K, V, table, q, kv_len, starts = build(rows, 8, 1, 128, 64, 64, 77, F32)
    c = gpu_cache(K, V, table)
    q, kv_len, starts = q.cuda(), kv_len.cuda(), starts.cuda()
    qs = [q * (1 + i) for i in range(4)]
    want = [c.attend(x, kv_len, starts, max_new=16) for x in qs]
    torch.cuda.synchronize()
    got = [[] for _ in qs]

    def work(i):
        for _ in range(50):
            got[i].append(c.attend(qs[i], kv_len, starts, max_new=16))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    c.check()
    assert [len(g) for g in got] == [50] * 4
    assert all(torch.equal(o, w) for g, w in zip(got, want) for o in g)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_recorded_prompts(dtype):
    """A recorded append and prompt attention (split over positions and not) replayed at other lengths and contents."""
    rows = [(1500, 40), (300, 33)]
    K, V, table, q, kv_len, starts = build(rows, 8, 2, 64, 64, 64, 31, dtype, poison=False)
    cache = gpu_cache(K, V, table)
    g = torch.Generator().manual_seed(6)
    k, v = (torch.randn(q.shape[0], 2, 64, generator=g).to(dtype) for _ in range(2))
    lens, st, qs, ks, vs = kv_len.cuda(), starts.cuda(), q.cuda(), k.cuda(), v.cuda()
    ws = torch.zeros(cache.workspace_bytes(q.shape[0], 8, 40, dtype=dtype), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(qs)
    gr, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(gr, stream=stream):
        cache.append(ks, vs, lens, q_start=st, max_new=40)
        cache.attend(qs, lens, q_start=st, max_new=40, out=out, workspace=ws)
    for now in ([(1500, 40), (300, 33)], [(800, 17), (70, 20)], [(40, 40), (0, 0)], [(1500, 1), (33, 33)]):
        starts = starts_of([n for _, n in now])
        lens.copy_(torch.tensor([l for l, _ in now], dtype=torch.int32))
        st.copy_(starts)
        out.fill_(5.0)
        gr.replay()
        torch.cuda.synchronize()
        for s, x in ((K, k), (V, v)):
            for r, (l, n) in enumerate(now):
                s.append(table[r], l - n, x[starts[r]:starts[r + 1]].double())
        compare(out, now, K, V, table, q, 0, 0, dtype)
        assert bool((out[int(starts[-1]):] == 5).all())
    cache.check()


@pytest.mark.parametrize("new", [1, 3, 40])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_bad_queries_keep_to_themselves(new, dtype):
    """NaN and infinities in one token's q: its heads' results are NaN, the others' as without them."""
    rows = [(100, new), (90, new)]
    K, V, table, q, kv_len, starts = build(rows, 8, 2, 64, 16, 16, 13, dtype)
    cache = gpu_cache(K, V, table)
    good = cache.attend(q.cuda(), kv_len.cuda(), q_start=starts.cuda(), max_new=new)
    for value in (math.nan, math.inf):
        bad = q.clone()
        bad[new - 1, 3, 7] = value
        bad[new, 5] = 0.0            # a row of zeros: the mean of what it sees
        out = cache.attend(bad.cuda(), kv_len.cuda(), q_start=starts.cuda(), max_new=new)
        assert bool(torch.isnan(out[new - 1, 3]).all())
        ok = torch.ones(out.shape[:2], dtype=torch.bool)
        ok[new - 1, 3] = ok[new, 5] = False
        assert torch.equal(out[ok.cuda()], good[ok.cuda()])
        o, mass, score = R.attend(bad[new:new + 1].double(), K.values(table[1].long()), V.values(table[1].long()), torch.tensor([90 - new]))
        lim = R.bound(mass, score, o, dtype, 64, 90)
        assert bool(((out[new].double().cpu() - o[0]).abs() <= lim[0])[5].all())
    cache.check()


def test_many_rows_and_the_smallest():
    """More rows than a warp has lanes, most of them idle; then one row of one position."""
    g = torch.Generator().manual_seed(2)
    n = 1024
    lens = torch.where(torch.rand(n, generator=g) < 0.1, torch.randint(1, 200, (n,), generator=g), torch.zeros(n, dtype=torch.long))
    lens[700], lens[1023] = 900, 1
    rows = [(int(l), 1) for l in lens]
    K, V, table, q, kv_len, _ = build(rows, 4, 2, 64, 64, 64, 3, F32, poison=False)
    cache = gpu_cache(K, V, table)
    out = cache.attend(q.cuda(), kv_len.cuda())
    cache.check()
    for r in [0, 31, 32, 700, 1022, 1023] + [r for r in range(n) if lens[r]][:40]:
        compare(out[r:r + 1], [rows[r]], K, V, table[r:r + 1], q[r:r + 1], 0, 0, F32)
    assert bool((out[(lens == 0).cuda()] == 0).all())


@pytest.mark.parametrize("heads,new,window", [(8, 5, 0), (8, 12, 0), (6, 7, 2100), (10, 6, 0), (8, 13, 0)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_drafts_of_a_large_batch(heads, new, window, dtype):
    """Drafts of more than 16 query rows, of unequal lengths, idle and short rows among them: 40 rows x 2 heads."""
    rows = [(7 * r + 2050 if r % 11 == 0 else 13 * r + 1, max(new - r % 4, 1)) for r in range(40)]
    rows[3], rows[8], rows[9], rows[20] = (0, new), (2, new), (4, 0), (new - 2, new)
    K, V, table, q, kv_len, starts = build(rows, heads, 2, 64, 64, 32, 91, dtype)
    c = gpu_cache(K, V, table)
    out = c.attend(q.cuda(), kv_len.cuda(), starts.cuda(), max_new=new, window=window, sinks=3 if window else 0)
    c.check()
    compare(out, rows, K, V, table, q, window or None, 3 if window else 0, dtype)


@pytest.mark.parametrize("new", [1, 64])
def test_repeats_bit_for_bit(new):
    rows = [(3000, new), (10 + new, new), (777, new)]
    K, V, table, q, kv_len, starts = build(rows, 8, 2, 128, 64, 64, 8, F32, poison=False)
    cache = gpu_cache(K, V, table)
    first = cache.attend(q.cuda(), kv_len.cuda(), q_start=starts.cuda(), max_new=new)
    for _ in range(5):
        assert torch.equal(first, cache.attend(q.cuda(), kv_len.cuda(), q_start=starts.cuda(), max_new=new))


@pytest.mark.parametrize("new", [1, 40])
def test_offsets_past_32_bits(new):
    """Pages at the end of pools of over 2^32 bytes."""
    from graph_replay_gb300 import KV8Cache
    heads, kv_heads, dim, page = 4, 2, 128, 64
    pages = (1 << 32) // (kv_heads * page * dim) + 100
    rows = [(200, new)]
    K, V, table, q, kv_len, starts = build(rows, heads, kv_heads, dim, page, 64, 6, F32)
    per = table.shape[1]
    (kb, ks), (vb, vs) = K.bytes(), V.bytes()
    big = torch.arange(pages - per, pages, dtype=torch.int32).view(1, per)
    ks_, vs_ = (torch.full((pages, kv_heads, 1), 127, dtype=torch.uint8, device="cuda") for _ in range(2))
    k_, v_ = (torch.empty(pages, kv_heads, page, dim, dtype=torch.uint8, device="cuda") for _ in range(2))
    at = table[0].long()
    k_[-per:], v_[-per:], ks_[-per:], vs_[-per:] = kb[at].cuda(), vb[at].cuda(), ks[at].cuda(), vs[at].cuda()
    cache = KV8Cache(k_, v_, ks_, vs_, page_table=big.cuda())
    out = cache.attend(q.cuda(), kv_len.cuda(), q_start=starts.cuda(), max_new=new)
    compare(out, rows, K, V, table, q, 0, 0, F32)
    k, v = torch.randn(1, kv_heads, dim), torch.randn(1, kv_heads, dim)
    cache.append(k.cuda(), v.cuda(), torch.tensor([201], dtype=torch.int32).cuda())
    K.append(table[0], 200, k.double())
    V.append(table[0], 200, v.double())
    out = cache.attend(q[:1].cuda(), torch.tensor([201], dtype=torch.int32).cuda())
    compare(out, [(201, 1)], K, V, table, q[:1], 0, 0, F32)
    cache.check()
    del cache, k_, v_
    torch.cuda.empty_cache()


def test_refusals_on_tensors():
    from graph_replay_gb300 import KV8Cache, _binding as B
    cache = KV8Cache.empty(2, 64, 2, 64)
    lens = torch.ones(2, dtype=torch.int32, device="cuda")
    q = torch.zeros(2, 4, 64, device="cuda")
    for bad in (q.half(), q[..., :32], q.cpu(), q.transpose(0, 1), q[:, :3]):
        with pytest.raises((ValueError, B.DecError)):
            cache.attend(bad, lens)
    with pytest.raises(ValueError):
        cache.attend(q, lens.long())
    with pytest.raises(ValueError):
        cache.attend(q, lens[:1])
    with pytest.raises(ValueError):
        cache.attend(q, lens, out=torch.zeros(2, 4, 64, device="cuda", dtype=BF16))
    with pytest.raises(B.DecError, match="q_start"):
        cache.attend(torch.zeros(3, 4, 64, device="cuda"), lens)
    with pytest.raises(B.DecError, match="window"):
        cache.attend(q, lens, window=-1)
    with pytest.raises(B.DecError, match="aligned"):
        cache.attend(torch.zeros(2 * 4 * 64 + 1, device="cuda")[1:].view(2, 4, 64), lens)
    with pytest.raises(ValueError):
        KV8Cache(cache.k, cache.v, cache.k_scale, cache.v_scale)
    with pytest.raises(ValueError):
        cache.append(q, q, lens)
    # nothing to do: no tokens at all
    none = torch.zeros(0, 4, 64, device="cuda")
    assert cache.attend(none, lens, q_start=torch.zeros(3, dtype=torch.int32, device="cuda")).shape == none.shape
