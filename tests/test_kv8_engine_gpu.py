"""Captures with an e4m3 K/V store: the step, its attention, the prefills and the window, against a plain fp64 decoder
that stores K and V by the same rules."""
import math

import numpy as np
import pytest
import torch

import _kv8 as R

pytestmark = pytest.mark.gpu
D, HEADS, KV, HD, F, VOCAB, LAYERS, THETA, EPS = 1024, 16, 4, 64, 1024, 512, 2, 1e4, 1e-5   # 2..8 bf16 rows take multiples of 1024


def weights(dtype, heads=HEADS, kv=KV, hd=HD, seed=0):
    g = torch.Generator().manual_seed(seed)

    def m(*shape, s=0.03):
        return (torch.randn(*shape, generator=g) * s).to(dtype)
    one = lambda: (1 + 0.1 * torch.randn(D, generator=g)).to(dtype)  # noqa: E731
    w = {"embed": m(VOCAB, D, s=1.0), "final_norm": one(), "lm_head": m(VOCAB, D), "layers": []}
    for _ in range(LAYERS):
        w["layers"].append({"attn_norm": one(), "wq": m(heads * hd, D), "wk": m(kv * hd, D), "wv": m(kv * hd, D),
                            "wo": m(D, heads * hd), "ffn_norm": one(), "wg": m(F, D), "wu": m(F, D), "wd": m(D, F)})
    return w


def on_gpu(w):
    return {k: [{n: t.cuda() for n, t in l.items()} for l in v] if k == "layers" else v.cuda() for k, v in w.items()}


def decoder(w, rows, cap, paged=False, page=16, dtype="bf16", heads=HEADS, kv=KV, hd=HD, **kw):
    from graph_replay_gb300 import Decoder, make_config
    cfg = make_config(LAYERS, D, heads, kv, hd, F, VOCAB, dtype, "e4m3", EPS, THETA, device=0)
    if paged:
        kw.update(kv_layout="paged", page_size=page, num_pages=rows * cap // page + 3)
    return Decoder(cfg, on_gpu(w), cap=cap, rows=rows, **kw)


def rope(x, pos):
    """x [tokens, heads, dim], pos [tokens]"""
    h = x.shape[-1] // 2
    a = pos.double()[:, None] * THETA ** (-2.0 * torch.arange(h).double() / x.shape[-1])
    c, s = torch.cos(a)[:, None], torch.sin(a)[:, None]
    return torch.cat([x[..., :h] * c - x[..., h:] * s, x[..., :h] * s + x[..., h:] * c], -1)


class Plain:
    """The decoder in fp64, one sequence; K and V as stored."""

    def __init__(self, w, cap, block, window=0, sinks=0):
        self.w = {k: [{n: t.double() for n, t in l.items()} for l in v] if k == "layers" else v.double() for k, v in w.items()}
        self.K, self.V = ([R.Store(1, KV, cap, HD, block) for _ in range(LAYERS)] for _ in range(2))
        self.window, self.sinks = window, sinks

    def run(self, tokens, pos0):
        """tokens at pos0, pos0 + 1, ...: K and V of all stored first, layer by layer; logits of the last."""
        pos = torch.arange(pos0, pos0 + len(tokens))
        x = self.w["embed"][torch.as_tensor(tokens).long()]
        norm = lambda y, g: y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * g  # noqa: E731
        for l, w in enumerate(self.w["layers"]):
            h = norm(x, w["attn_norm"])
            q, k, v = ((h @ w[n].T).view(len(tokens), -1, HD) for n in ("wq", "wk", "wv"))
            self.K[l].append([0], pos0, rope(k, pos))
            self.V[l].append([0], pos0, v)
            row = torch.tensor([0])
            o, _, _ = R.attend(rope(q, pos), self.K[l].values(row), self.V[l].values(row), pos, self.window, self.sinks)
            x = x + o.flatten(1) @ w["wo"].T
            h = norm(x, w["ffn_norm"])
            g = h @ w["wg"].T
            x = x + (g * torch.sigmoid(g) * (h @ w["wu"].T)) @ w["wd"].T
        return (norm(x[-1:], self.w["final_norm"]) @ self.w["lm_head"].T)[0].numpy()


# The GPU's k and v carry fp32 (bf16 rows >= 2: 16-bit hi + lo operand) errors, so a value next to a rounding border may
# be stored one e4m3 step (2^-3 of itself) away.  Such a step in k moves a score by at most 2^-3 |q_d k_d| / 8, about a
# hundredth, and its weight by as much; in v it moves one of 64 dims of one weight's share.  A few of them stay below
# 2e-2 of a head's result, and the residual stream dilutes that; a wrong position, scale or mask is of order one.
STEP_TOL = 2e-2


def near(got, ref, what):
    off = float(np.linalg.norm(got - ref) / np.linalg.norm(ref))
    assert np.isfinite(got).all() and off <= STEP_TOL, f"{what}: {off:.3g}"


def slot_map(dec, rows, cap, page, seed=3):
    m = np.random.RandomState(seed).permutation(dec.num_pages)[:rows * cap // page].reshape(rows, -1).astype(np.int32)
    dec.set_slot_map(m)
    return m


@pytest.mark.parametrize("dtype,rows,paged,window,sinks", [("f32", 1, False, 0, 0), ("f32", 3, True, 0, 0), ("bf16", 1, True, 7, 2),
                                                            ("bf16", 4, False, 0, 0), ("bf16", 8, True, 5, 0)])
def test_steps(dtype, rows, paged, window, sinks):
    cap, w = 64, weights(torch.float32 if dtype == "f32" else torch.bfloat16)
    dec = decoder(w, rows, cap, paged, 16, dtype, window=window, sinks=sinks)
    if paged:
        slot_map(dec, rows, cap, 16)
    ref = [Plain(w, cap, 16 if paged else 64, window, sinks) for _ in range(rows)]
    rng = np.random.RandomState(1)
    # each row from its own position on: rows cross block borders at different steps
    at = [3 * r for r in range(rows)]
    for r in range(rows):
        for p in range(at[r]):
            ref[r].run([0], p)
    for p in range(max(at)):   # the others repeat position 0 meanwhile
        dec.step([0] * rows, [min(p, a - 1) if a else 0 for a in at])
    for i in range(24):
        tok = rng.randint(0, VOCAB, rows)
        res = dec.step(tok, at)
        for r in range(rows):
            near(res.logits[r], ref[r].run([int(tok[r])], at[r]), f"step {i} row {r}")
            at[r] += 1
    st = dec.stats()
    assert st["replays"] == 24 + (max(at) - 24) and st["last_fault"] == 0
    dec.close()


def test_replay_equals_eager_and_chain():
    w = weights(torch.bfloat16)
    ids = []
    for eager in (False, True):
        dec = decoder(w, 2, 64, window=9, sinks=1)
        dec.set_eager(eager)
        out = [dec.step([5 + i, 9 + i], [i, i]) for i in range(20)]
        ids.append([(o.logits.copy(), o.ids.copy()) for o in out])
        dec.reset_state()
        chain, nf = dec.chain([5, 9], [0, 0], 12)
        assert not nf.any()
        dec.reset_state()
        tok = [5, 9]
        for i in range(12):
            tok = dec.step(tok, [i, i]).ids
            assert (tok == chain[i]).all()
        dec.close()
    for a, b in zip(*ids):
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("n,window,sinks", [(1, 0, 0), (5, 0, 0), (37, 0, 0), (150, 0, 0), (150, 20, 3)])
def test_block_prefill_then_steps(paged, n, window, sinks):
    cap, w = 192, weights(torch.bfloat16)
    dec = decoder(w, 2, cap, paged, 32, window=window, sinks=sinks)
    pages = slot_map(dec, 2, cap, 32)[1] if paged else None
    tok = np.random.RandomState(2).randint(0, VOCAB, n + 6)
    ref = Plain(w, cap, 32 if paged else 64, window, sinks)
    first = n // 2 + 1   # two calls: the second continues behind the first
    for a, b in ((0, first), (first, n)):
        if b > a:
            logits, _ = dec.prefill_block(tok[a:b], pos0=a, row=1, pages=pages)
            near(logits, ref.run(list(tok[a:b]), a), f"prefill to {b}")
    for p in range(n, n + 6):
        res = dec.step([0, tok[p]], [0, p])
        near(res.logits[1], ref.run([int(tok[p])], p), f"step {p}")
    dec.close()


def test_block_prefill_any_group_and_long():
    """Groups of 8 (the bf16 store's prefill takes 2 and 4) and more than one pass of 1024 tokens agree with single steps' store."""
    from graph_replay_gb300 import Decoder, make_config
    w = weights(torch.bfloat16, heads=8, kv=1)
    dec = decoder(w, 1, 1280, heads=8, kv=1, window=100, sinks=4)
    tok = np.random.RandomState(5).randint(0, VOCAB, 1100)
    logits, _ = dec.prefill_block(tok[:1099])
    a = dec.step([tok[1099]], [1099]).logits[0]
    other = decoder(w, 1, 1280, heads=8, kv=1, window=100, sinks=4)
    other.prefill_block(tok[:1000])
    for p in range(1000, 1100):
        b = other.step([tok[p]], [p]).logits[0]
        if p == 1098:
            near(logits, b, "the prefill's own logits")
    near(a, b, "a step after it")
    dec.close(), other.close()


def test_chunked_prefill_shares_blocks():
    cap, w = 64, weights(torch.bfloat16)
    dec = decoder(w, 4, cap, True, 32)
    pages = slot_map(dec, 4, cap, 32)[2]
    tok = np.random.RandomState(4).randint(0, VOCAB, 30)
    ref = Plain(w, cap, 32)
    logits, _ = dec.prefill(pages, tok[:27])
    for p in range(0, 27, 4):   # chunks of the capture's rows
        out = ref.run(list(tok[p:min(p + 4, 27)]), p)
    near(logits, out, "chunked prefill")
    for p in range(27, 30):
        res = dec.step([0, 0, tok[p], 0], [0, 0, p, 0])
        near(res.logits[2], ref.run([int(tok[p])], p), f"step {p}")
    dec.close()


@pytest.mark.parametrize("paged,rows,hd,heads,kv,window,sinks", [(False, 1, 128, 4, 1, 0, 0), (True, 4, 64, 8, 2, 33, 5), (False, 8, 64, 2, 2, 0, 0)])
def test_attention_on_the_store(paged, rows, hd, heads, kv, window, sinks):
    """dec_attention on a store filled by hand: what is stored, and the result for exactly what is stored."""
    cap = 320
    w = weights(torch.float32, heads, kv, hd)
    dec = decoder(w, rows, cap, paged, 64, "f32", heads, kv, hd, window=window, sinks=sinks)
    m = slot_map(dec, rows, cap, 64) if paged else np.arange(rows)[:, None].astype(np.int32)
    g = torch.Generator().manual_seed(8)
    ks, vs, kx, vx = dec.kv_scale(1, 0), dec.kv_scale(1, 1), dec.kv(1, 0), dec.kv(1, 1)
    for x, s in ((kx, ks), (vx, vs)):
        x.copy_((torch.randn(x.shape, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn))
        s.copy_(torch.randint(119, 124, s.shape, generator=g, dtype=torch.uint8))
    pos = torch.tensor([(97 * r + 203) % cap for r in range(rows)], dtype=torch.int32)
    qkv = torch.randn(rows, (heads + 2 * kv) * hd, generator=g)
    if paged:   # the write map is a slot of its own: a step sets it
        dec.step([0] * rows, pos.tolist())
    out = torch.empty(rows, heads * hd, device="cuda")
    before = [t.float().cpu() for t in (kx, vx)], [t.cpu().clone() for t in (ks, vs)]
    dec.attention(1, qkv.cuda(), pos.cuda(), out)
    page = 64 if paged else cap
    for which, x, s in ((0, kx, ks), (1, vx, vs)):
        st = R.Store(x.shape[0], kv, page, hd, 64)
        st.x, st.e = before[0][which].double(), before[1][which].long() - 127
        for r in range(rows):
            new = qkv[r, (heads + which * kv) * hd:(heads + (which + 1) * kv) * hd].double().view(1, kv, hd)
            st.append(torch.as_tensor(m[r]), int(pos[r]), rope(new, pos[r:r + 1]) if which == 0 else new)
        got, want = x.float().cpu().double(), st.x
        assert torch.equal(s.cpu().long() - 127, st.e)
        assert bool(((got - want).abs() <= want.abs() * 2.0 ** -3 + 2.0 ** -9).all()) and int((got != want).sum()) <= 3 * rows
        st.x = got
        if which == 0:
            K = st
        else:
            V = st
    for r in range(rows):
        p = pos[r:r + 1].long()
        q = rope(qkv[r:r + 1, :heads * hd].double().view(1, heads, hd), p)
        row = torch.as_tensor(m[r]).long()
        o, mass, score = R.attend(q, K.values(row), V.values(row), p, window, sinks)
        # the GPU's q after RoPE is off by an fp32 product and sum: 2^-22 of the score more than the bound has
        lim = R.bound(mass, score, o, torch.float32, hd, cap) + mass * score * 2.0 ** -21
        off = (out[r].cpu().double().view(1, heads, hd) - o).abs()
        assert bool((off <= lim).all()), f"row {r}: {float((off / lim).max()):.3g} of what the arithmetic allows"
    dec.close()


def test_faults_and_refusals():
    from graph_replay_gb300 import Decoder, make_config, _binding as B
    w = weights(torch.bfloat16)
    dec = decoder(w, 2, 64, True, 16)
    good = dec.step([1, 2], [0, 0]).logits.copy()
    # the device's own checks: WriteMap behind the pool, then a position behind the capacity
    for slots, bit in (([1, 2, 1, 1, 1, 10 ** 6], 0x4), ([1, 2, 1, 64, 1, 1], 0x2)):
        dec.launch(torch.tensor(slots, dtype=torch.int32, device="cuda"))
        with pytest.raises(B.DecError) as e:
            dec.wait()
        assert e.value.status == B.DEC_E_DEVICE_FAULT and dec.stats()["last_fault"] & bit
        dec.reset_state()
        assert np.array_equal(dec.step([1, 2], [0, 0]).logits, good)
        dec.reset_state()
    # the fixed array of dec_attention_static is not for this store; the handle stays usable
    buf = torch.zeros(2, (HEADS + 2 * KV) * HD, device="cuda")
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert B.dec_attention_static(dec.h, 0, buf.data_ptr(), pos.data_ptr(), buf.data_ptr()) == B.DEC_E_UNSUPPORTED
    assert np.array_equal(dec.step([1, 2], [0, 0]).logits, good)
    with pytest.raises(B.DecError, match="before dec_capture"):
        B.dec_set_window(dec.h, 4, 0)
    dec.close()
    cfg = lambda kv, **k: make_config(LAYERS, D, HEADS, KV, HD, F, VOCAB, "bf16", kv, EPS, THETA)  # noqa: E731
    for kw, word, kvt in ((dict(cap=60), "multiple of 16", "e4m3"), (dict(cap=64, kv_layout="paged", page_size=8, num_pages=32), "16", "e4m3"),
                          (dict(cap=64, strategy="persistent"), "GRAPH", "e4m3"), (dict(cap=64, window=5), "window", "bf16")):
        with pytest.raises(B.DecError, match=word) as e:
            Decoder(cfg(kvt), on_gpu(w), rows=1, lib_workspace=True, **kw)
        assert e.value.status == B.DEC_E_UNSUPPORTED
    d = Decoder(cfg("bf16"), on_gpu(w), rows=1, cap=64)
    with pytest.raises(B.DecError, match="scales"):
        d.kv_scale(0, 0)
    d.close()


@pytest.mark.parametrize("at", [[0, 1, 2, 3], [3, 2, 1, 0], [37, 32, 41, 34], [60, 5, 61, 4], [50, 50, 7, 50], [15, 16, 0, 31]], ids=str)
@pytest.mark.parametrize("hd,page", [(64, 64), (128, 32), (64, 16)])
def test_rows_that_share_blocks_in_any_order(at, hd, page):
    """Rows of one sequence step at positions in any order, with values far apart: one scale a block, from all of them;
    what the block held below the last of them is rounded again; of equal positions the last row's counts."""
    heads, kv, cap, rows, block = 4, 2, 64, 4, page
    w = weights(torch.float32, heads, kv, hd)
    dec = decoder(w, rows, cap, True, page, "f32", heads, kv, hd)
    pages = [2, 0, 3, 1][:cap // page]
    dec.set_slot_map(np.array([pages] * rows, dtype=np.int32))
    g = torch.Generator().manual_seed(3)
    dec.step([0] * rows, at)   # the write map
    stores = [(dec.kv(0, i), dec.kv_scale(0, i)) for i in (0, 1)]
    for x, s in stores:
        x.copy_((torch.randn(x.shape, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn))
        s.copy_(torch.randint(119, 122, s.shape, generator=g, dtype=torch.uint8))
    before = [(x.float().cpu().double(), s.cpu().long() - 127) for x, s in stores]
    qkv = torch.randn(rows, (heads + 2 * kv) * hd, generator=g) * (8.0 ** torch.arange(rows))[torch.randperm(rows, generator=g), None]
    pos, out = torch.tensor(at, dtype=torch.int32), torch.empty(rows, heads * hd, device="cuda")
    dec.attention(0, qkv.cuda(), pos.cuda(), out)
    torch.cuda.synchronize()
    counts = [r for r in range(rows) if at[r] not in at[r + 1:]]
    for which in (0, 1):
        x, e = (t.clone() for t in before[which])
        new = qkv[:, (heads + which * kv) * hd:(heads + (which + 1) * kv) * hd].double().view(rows, kv, hd)
        new = rope(new, pos) if which == 0 else new
        for b in {at[r] // block for r in counts}:
            here = [r for r in counts if at[r] // block == b]
            pg, first = pages[b * block // page], b * block % page
            for h in range(kv):
                held = [j for j in range(max(at[r] for r in here) % block) if b * block + j not in at]
                was, need = int(e[pg, h, first // block]), R.exponent(float(new[here, h].abs().max()))
                e[pg, h, first // block] = now = max(was, need) if held else need
                for j in held:
                    x[pg, h, first + j] = R.e4m3(x[pg, h, first + j] * 2.0 ** (was - now))
                for r in here:
                    x[pg, h, first + at[r] % block] = R.e4m3(new[r, h] * 2.0 ** -now)
        got, scale = stores[which][0].float().cpu().double(), stores[which][1].cpu().long() - 127
        assert torch.equal(scale, e)
        if which == 1:
            assert torch.equal(got, x)
        else:   # k after RoPE carries fp32 errors: a value next to a rounding border may be stored a step away
            assert bool(((got - x).abs() <= x.abs() * 2.0 ** -3 + 2.0 ** -9).all()) and int((got != x).sum()) <= 3 * rows
    dec.close()


@pytest.mark.parametrize("paged", [False, True])
def test_stats_count_the_scales(paged):
    w = weights(torch.bfloat16)
    dec = decoder(w, 2, 256, paged, 16)
    parts = [t.numel() for l in range(LAYERS) for i in (0, 1) for t in (dec.kv(l, i), dec.kv_scale(l, i))]
    assert sum(parts) <= dec.stats()["kv_bytes"] <= sum(parts) + 256 * len(parts)   # each part up to a multiple of 256
    dec.close()
