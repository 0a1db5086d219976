"""Captures whose matrices are bound in 4 bits, against the oracle over the values that they stand for."""
import dataclasses

import numpy as np
import pytest
import torch

import gen
import oracle
from _harness import assert_close, assert_greedy

pytestmark = pytest.mark.gpu
MATRICES = ("wq", "wk", "wv", "wo", "wg", "wu", "wd")


def as_f32(a):
    return gen.bf16_bits_to_f32(a) if a.dtype == np.uint16 else a


def stored(wl, group=128, head=True, seed=None):
    """(weights for the decoder, the oracle's model) of a workload: its matrices, and with `head` the LM head, in 4 bits."""
    from gen.device import upload_weights
    from graph_replay_gb300 import W4Weight
    mw = gen.make_weights(wl)
    w = upload_weights(mw, "cuda:0")
    ref = dataclasses.replace(mw, wl=wl.replace(wdtype="f32"), embed=as_f32(mw.embed), final_norm=as_f32(mw.final_norm),
                              lm_head=as_f32(mw.lm_head), layers=[{k: as_f32(v) for k, v in l.items()} for l in mw.layers])
    for lw, rl in zip(w["layers"], ref.layers):
        for name in MATRICES:
            lw[name] = W4Weight.quantize(lw[name], group)
            rl[name] = lw[name].dequantize().cpu().numpy()
    if head:
        w["lm_head"] = W4Weight.quantize(w["lm_head"], group)
        ref.lm_head = w["lm_head"].dequantize().cpu().numpy()
    return w, ref


def decoder(wl, w, **kw):
    from graph_replay_gb300 import Decoder, make_config
    cfg = make_config(wl.n_layers, wl.d_model, wl.n_heads, wl.n_kv_heads, wl.head_dim, wl.ffn_hidden, wl.vocab, wl.wdtype,
                      kw.pop("kv_dtype", wl.kvdtype), wl.rms_eps, wl.rope_theta, device=0)
    return Decoder(cfg, w, cap=wl.cap, rows=wl.rows, kv_layout=wl.layout, page_size=wl.page_size, num_pages=wl.num_pages, **kw)


def check_steps(wl, w, ref, steps, **kw):
    """Every row its own sequence, from positions apart; logits, ids and flags of each step."""
    dec = decoder(wl, w, **kw)
    orcs = [oracle.Oracle(ref, cap=wl.cap) for _ in range(wl.rows)]
    toks = [gen.prompt_tokens(wl, row=r, n=steps) for r in range(wl.rows)]
    for i in range(steps):
        pos = [i + 3 * r for r in range(wl.rows)]
        res = dec.step([int(t[i]) for t in toks], pos)
        for r in range(wl.rows):
            want = orcs[r].step(0, int(toks[r][i]), pos[r])
            # fp32 throughout but for the K/V store: its rounding decides the tolerance
            assert_close(res.logits[r], want, wl.replace(wdtype="f32" if wl.kvdtype == "f32" else "bf16"), f"step {i} row {r}")
            assert_greedy(res.ids[r], want)
            assert res.nonfinite[r] == 0 and int(res.ids[r]) == int(np.argmax(res.logits[r]))
    dec.close()


@pytest.mark.parametrize("group", [32, 64])
@pytest.mark.parametrize("rows", [1, 3])
def test_tiny_model(group, rows):
    wl = gen.WORKLOADS["tiny_gain"].replace(rows=rows)
    check_steps(wl, *stored(wl, group), steps=12)


@pytest.mark.parametrize("rows, group, head", [(1, 128, True), (1, 32, False), (2, 64, True), (4, 128, False), (8, 128, True),
                                               (8, 32, True)])
def test_1b_shape(rows, group, head):
    wl = gen.WORKLOADS["1b"].replace(name="1b_w4", n_layers=2, cap=128, rows=rows, vocab=1003, gain_sigma=0.1)
    check_steps(wl, *stored(wl, group, head), steps=4)


def test_8b_layer():
    """The widest matrices: QKV stacked over 6144 rows, the block of 14336."""
    wl = gen.WORKLOADS["8b"].replace(name="8b_w4", n_layers=1, cap=64, rows=8, vocab=512)
    check_steps(wl, *stored(wl), steps=2)


def test_paged_prefill_chunks_then_decode():
    wl = gen.WORKLOADS["1b"].replace(name="1b_w4p", n_layers=2, cap=64, rows=8, vocab=512, layout="paged", page_size=16,
                                     num_pages=40)
    w, ref = stored(wl)
    dec = decoder(wl, w)
    table = gen.permutation(wl.seed, 5, wl.num_pages)[:8 * 4].reshape(8, 4).astype(np.int32)
    dec.set_slot_map(table)
    toks = [int(t) for t in gen.prompt_tokens(wl, n=21)]
    logits, _ = dec.prefill(table[2], toks)
    orc = oracle.Oracle(ref, cap=wl.cap)
    for p, t in enumerate(toks):
        want = orc.step(0, t, p)
    assert_close(logits, want, wl, "after the prompt")
    nxt = int(np.argmax(want))
    res = dec.step([0, 0, nxt] + [0] * 5, [0, 0, 21] + [0] * 5)
    assert_close(res.logits[2], orc.step(0, nxt, 21), wl, "the step after it")
    dec.close()


def test_replay_eager_and_chain_agree():
    wl = gen.WORKLOADS["1b"].replace(name="1b_w4c", n_layers=2, cap=64, rows=2, vocab=512)
    w, _ = stored(wl)
    dec = decoder(wl, w)
    a = [dec.step([5, 9], [i, i]) for i in range(3)]
    dec.reset_state()
    dec.set_eager(True)
    b = [dec.step([5, 9], [i, i]) for i in range(3)]
    dec.set_eager(False)
    for x, y in zip(a, b):
        assert np.array_equal(x.logits, y.logits) and np.array_equal(x.ids, y.ids)
    dec.reset_state()
    ids, nf = dec.chain([5, 9], [0, 0], 6)
    dec.reset_state()
    tok = [5, 9]
    for i in range(6):
        tok = dec.step(tok, [i, i]).ids
        assert np.array_equal(tok, ids[i])
    assert not nf.any()
    dec.close()


def test_with_an_8_bit_store_and_a_sampler():
    """Both 8-bit K/V and 4-bit matrices: near the same model with a bf16 store; picks are the sampler's at temperature 0."""
    wl = gen.WORKLOADS["1b"].replace(name="1b_w4k", n_layers=2, cap=64, rows=2, vocab=512)
    w, _ = stored(wl)
    a, b = decoder(wl, w), decoder(wl, w, kv_dtype="e4m3", sampler=dict(temperature=0.0, n_logprobs=2))
    for i in range(5):
        x, y = a.step([7, 11], [i, i]), b.step([7, 11], [i, i])
        assert np.linalg.norm(x.logits - y.logits) <= 0.1 * np.linalg.norm(x.logits)   # e4m3 keeps 4 bits of K and V
        assert np.array_equal(y.ids, y.logits.argmax(-1))
        ids, _ = b.logprobs(2)
        assert np.array_equal(ids[:, 0], y.ids)
    a.close()
    b.close()


def test_kernels_alone_and_bytes():
    from graph_replay_gb300 import _binding as B
    wl = gen.WORKLOADS["1b"].replace(name="1b_w4b", n_layers=1, cap=64, rows=1, vocab=512)
    w, _ = stored(wl)
    dec = decoder(wl, w)
    dec.step([1], [0])
    d, f = wl.d_model, wl.ffn_hidden
    n = B.dec_launch_kernel(dec.h, 4)   # gate/up
    assert n == 2 * f * d // 2 + 2 * (2 * f * d // 128) + d * 4 + f * 4 + d * 2
    dec.close()


def test_refusals():
    from graph_replay_gb300 import W4Weight
    from graph_replay_gb300 import _binding as B
    wl = gen.WORKLOADS["1b"].replace(name="1b_w4r", n_layers=1, cap=64, rows=1, vocab=512)
    w, _ = stored(wl)
    for mend, word in ((lambda l: l.update(wk=l["wk"].dequantize(torch.bfloat16)), "all seven"),
                       (lambda l: l.update(wv=W4Weight.quantize(l["wv"].dequantize(), 64)), "one group"),
                       (lambda l: l.update(wu=W4Weight.quantize(l["wu"].dequantize(), 32)), "one group"),
                       (lambda l: l.update(wo=l["wk"]), "shape"),
                       (lambda l: l.update(ffn_norm=l["wq"]), "no 4-bit form")):
        bad = dict(w, layers=[dict(l) for l in w["layers"]])
        mend(bad["layers"][0])
        with pytest.raises(B.DecError, match=word):
            decoder(wl, bad)
    with pytest.raises(B.DecError, match="persistent"):
        decoder(wl, w, strategy="persistent")
    dec = decoder(wl, w)
    with pytest.raises(B.DecError, match="block prefill"):
        dec.prefill_block([1, 2, 3])
    with pytest.raises(B.DecError, match="before dec_capture"):
        B.dec_load_w4(dec.h, [B.dec_w4_binding(B.DEC_W_LM_HEAD, -1, w["lm_head"]._c)])
    dec.step([3], [0])   # still usable
    dec.close()
