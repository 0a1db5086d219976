"""Captures with some matrices in 4 bits and the others as they are: a head alone, some of the layers, each its own groups."""
import dataclasses

import numpy as np
import pytest

import gen
import oracle
from _harness import assert_close, assert_greedy
from test_w4_engine_gpu import MATRICES, as_f32, check_steps, decoder

pytestmark = pytest.mark.gpu


def mixed(wl, groups, head):
    """groups: of each layer, or None for one that stays as it is; head: the LM head's group or None."""
    from gen.device import upload_weights
    from graph_replay_gb300 import W4Weight
    mw = gen.make_weights(wl)
    w = upload_weights(mw, "cuda:0")
    ref = dataclasses.replace(mw, wl=wl.replace(wdtype="f32"), embed=as_f32(mw.embed), final_norm=as_f32(mw.final_norm),
                              lm_head=as_f32(mw.lm_head), layers=[{k: as_f32(v) for k, v in l.items()} for l in mw.layers])
    for lw, rl, group in zip(w["layers"], ref.layers, groups):
        for name in MATRICES if group else ():
            lw[name] = W4Weight.quantize(lw[name], group)
            rl[name] = lw[name].dequantize().cpu().numpy()
    if head:
        w["lm_head"] = W4Weight.quantize(w["lm_head"], head)
        ref.lm_head = w["lm_head"].dequantize().cpu().numpy()
    return w, ref


@pytest.mark.parametrize("rows", [1, 4, 8])
@pytest.mark.parametrize("groups, head", [((64, None, 32), None), ((None, 128, None), 64)])
def test_some_layers(rows, groups, head):
    wl = gen.WORKLOADS["1b"].replace(name="1b_w4m", n_layers=3, cap=64, rows=rows, vocab=771, gain_sigma=0.1)
    check_steps(wl, *mixed(wl, groups, head), steps=3)


@pytest.mark.parametrize("rows", [1, 3])
def test_block_prefill_before_a_head_in_4_bits(rows):
    wl = gen.WORKLOADS["1b"].replace(name="1b_w4h", n_layers=2, cap=256, rows=rows, vocab=1003)
    w, ref = mixed(wl, (None, None), 64)
    dec = decoder(wl, w)
    toks = [int(t) for t in gen.prompt_tokens(wl, n=150)]
    logits, pick = dec.prefill_block(toks, 0, row=rows - 1)
    want = oracle.Oracle(ref, cap=wl.cap, alloc_kv=False).full_causal(np.asarray(toks, dtype=np.int32))[0][-1]
    assert_close(logits, want, wl, "after the prompt")
    assert_greedy(pick, want)
    dec.close()
