"""dec_w4_workspace reads sizes and types: a caller sizes its memory before it has any."""
import ctypes

import pytest
import torch

from test_w4_cpu import B, call, weight   # noqa: F401  (B is a fixture)

NONE = dict(x=None, out=None, err=None, x_stride=0, out_stride=0)
DEC_E_CUDA = 5


def ask(B, **kw):   # noqa: F811
    size = ctypes.c_size_t(7)
    return B.lib().dec_w4_workspace(weight(B), kw.pop("up", None), call(B, **kw), size), size.value


@pytest.mark.parametrize("kw", [dict(), dict(tokens=100), dict(tokens=100, gain=8), dict(tokens=40, x_dtype=1, out_dtype=1)])
def test_no_tensors(B, kw):   # noqa: F811
    """Every check passes: what answers is the plan, or without a GPU the device that is not there."""
    rc, size = ask(B, **NONE, **kw)
    assert rc == (0 if torch.cuda.is_available() else DEC_E_CUDA), B.last_error(None)
    assert ask(B, **NONE, up=weight(B), **kw)[0] == rc
    if rc == 0:
        assert size == ask(B, **kw)[1]


def test_overlaps_do_not_count(B):   # noqa: F811
    c = dict(out=1 << 20)   # x itself
    assert ask(B, **c)[0] == (0 if torch.cuda.is_available() else DEC_E_CUDA)


@pytest.mark.parametrize("kw, word", [(dict(tokens=-1), "tokens"), (dict(x_dtype=3), "x_dtype"), (dict(out_dtype=3), "out_dtype"),
                                      (dict(gain=16, gain_dtype=9), "gain"), (dict(gain=16, eps=-1.0), "eps")])
def test_bad_sizes_and_types(B, kw, word):   # noqa: F811
    assert ask(B, **NONE, **kw)[0] == 1 and word in B.last_error(None)
    assert ask(B, **NONE, up=weight(B), act=5)[0] == 1 and "act" in B.last_error(None)


def test_no_tokens(B):   # noqa: F811
    assert ask(B, **NONE, tokens=0) == (0, 0)
