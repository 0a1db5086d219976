"""The 8-bit K/V cache without a GPU: what its calls refuse, before any device call, and the tests' own definitions."""
import ctypes
import math

import pytest
import torch

import _kv8 as R


@pytest.fixture(scope="module")
def B():
    from graph_replay_gb300 import build, _binding
    build.build()
    return _binding


PTR = 1 << 20   # a 16-byte aligned address that is never read: the checks come first


def parts(B, cache={}, batch={}, attn={}, new={}):
    c = dict(k=PTR, v=PTR, k_scale=PTR, v_scale=PTR, pages=PTR, rows=2, pages_per_row=4, page_size=64, num_pages=8,
             n_kv_heads=2, head_dim=64, scale_block=64, device=0)
    b = dict(q_start=PTR, kv_len=PTR, err=PTR, total=5, max_new=3)
    a = dict(q=PTR, out=PTR, q_stride=256, out_stride=256, dtype=0, n_heads=4, window=0, sinks=0, scale=0.0)
    n = dict(k=PTR, v=PTR, k_stride=128, v_stride=128, dtype=0)
    c.update(cache), b.update(batch), a.update(attn), n.update(new)
    return B.dec_kv8_cache(**c), B.dec_kv8_batch(**b), B.dec_kv8_attn(**a), B.dec_kv8_new(**n)


CACHE = [(dict(k=None), 1, "required"), (dict(v_scale=None), 1, "required"), (dict(v=PTR + 8), 1, "aligned"),
         (dict(rows=0), 1, "rows"), (dict(rows=1025), 2, "rows"), (dict(head_dim=96), 2, "head_dim"),
         (dict(scale_block=8), 2, "scale_block"), (dict(scale_block=48), 2, "scale_block"),
         (dict(page_size=32), 1, "page_size"), (dict(page_size=0), 1, "page_size"), (dict(n_kv_heads=0), 1, "n_kv_heads"),
         (dict(pages_per_row=1 << 25), 2, "2^30"), (dict(pages=None, num_pages=7), 1, "num_pages"), (dict(device=-1), 1, "device")]
BATCH = [(dict(kv_len=None), 1, "kv_len"), (dict(err=None), 1, "err"), (dict(total=-1), 1, "total"), (dict(max_new=0), 1, "max_new"),
         (dict(q_start=None), 1, "q_start"), (dict(max_new=1 << 25), 2, "max_new")]


@pytest.mark.parametrize("what, code, word", CACHE)
def test_bad_caches(B, what, code, word):
    c, b, a, n = parts(B, cache=what)
    size = ctypes.c_size_t()
    for rc in (B.lib().dec_kv8_append(c, b, n, None), B.lib().dec_kv8_attend(c, b, a, None), B.lib().dec_kv8_workspace(c, b, a, size)):
        assert rc == code and word in B.last_error(None)


@pytest.mark.parametrize("what, code, word", BATCH)
def test_bad_batches(B, what, code, word):
    c, b, a, n = parts(B, batch=what)
    for rc in (B.lib().dec_kv8_append(c, b, n, None), B.lib().dec_kv8_attend(c, b, a, None)):
        assert rc == code and word in B.last_error(None)


@pytest.mark.parametrize("what, code, word", [
    (dict(q=None), 1, "q"), (dict(out=PTR + 4), 1, "out"), (dict(q_stride=255), 1, "stride"), (dict(out_stride=258), 1, "stride"),
    (dict(q_stride=-256), 1, "stride"), (dict(dtype=2), 1, "dtype"), (dict(n_heads=3), 1, "n_heads"), (dict(n_heads=258), 2, "128"),
    (dict(window=-1), 1, "window"), (dict(sinks=-1), 1, "sinks"), (dict(scale=-1.0), 1, "scale"), (dict(scale=math.nan), 1, "scale"),
    (dict(scale=1e300), 1, "scale")])
def test_bad_attention(B, what, code, word):
    c, b, a, _ = parts(B, attn=what)
    assert B.lib().dec_kv8_attend(c, b, a, None) == code and word in B.last_error(None)


@pytest.mark.parametrize("what, word", [(dict(k=None), "k"), (dict(v=PTR + 2), "aligned"), (dict(k_stride=127), "stride"), (dict(dtype=7), "dtype")])
def test_bad_tokens(B, what, word):
    c, b, _, n = parts(B, new=what)
    assert B.lib().dec_kv8_append(c, b, n, None) == B.DEC_E_INVALID and word in B.last_error(None)


def test_null_structs(B):
    c, b, a, n = parts(B)
    L = B.lib()
    for rc in (L.dec_kv8_append(None, b, n, None), L.dec_kv8_append(c, None, n, None), L.dec_kv8_append(c, b, None, None),
               L.dec_kv8_attend(c, b, None, None), L.dec_kv8_workspace(c, b, a, None)):
        assert rc == B.DEC_E_INVALID


def test_no_tokens_is_no_work(B):
    # nothing is launched, so nothing needs a device
    c, b, a, n = parts(B, batch=dict(total=0))
    assert B.lib().dec_kv8_append(c, b, n, None) == B.DEC_OK
    assert B.lib().dec_kv8_attend(c, b, a, None) == B.DEC_OK


# ---- the tests' definitions, against torch and closed forms ----

def test_e4m3_definition_is_torchs():
    x = torch.cat([torch.linspace(-448, 448, 20011), torch.randn(4096) * 0.02, torch.tensor([2.0 ** -10, 3 * 2.0 ** -10, 0.0])]).double()
    assert torch.equal(R.e4m3(x), x.float().to(torch.float8_e4m3fn).double())   # linspace and randn are fp32 values: exact


def test_exponent_is_least():
    assert R.exponent(0.0) == R.LOW and R.exponent(448.0) == 0 and R.exponent(448.0001) == 1 and R.exponent(1e38) == R.HIGH
    assert R.exponent(224.0) == -1


def test_growing_a_block_rounds_its_earlier_tokens():
    s = R.Store(1, 1, 16, 64, 16)
    one = torch.full((1, 1, 64), 1.0, dtype=torch.float64)
    s.append([0], 0, one)
    s.append([0], 1, one * 1000.0)
    assert int(s.e[0, 0, 0]) == 2                              # 1000 <= 448 * 4
    assert torch.equal(s.values(torch.tensor([0]))[0, 0], one[0, 0])   # a power of two shifts without loss
    s.append([0], 2, one * 2.0 ** 18)
    assert float(s.values(torch.tensor([0]))[0, 0, 0]) == 0.0 or abs(float(s.values(torch.tensor([0]))[0, 0, 0]) - 1.0) <= 1.0


def test_attention_definition_small_cases():
    k = torch.zeros(1, 4, 64, dtype=torch.float64)
    v = torch.arange(4.0).double()[None, :, None].expand(1, 4, 64)
    q = torch.ones(3, 2, 64, dtype=torch.float64)
    out, _, _ = R.attend(q, k, v, torch.tensor([-1, 1, 3]))
    assert out[:, 0, 0].tolist() == [0.0, 0.5, 1.5]
    out, _, _ = R.attend(q, k, v, torch.tensor([0, 2, 3]), window=1, sinks=1)
    assert out[:, 0, 0].tolist() == [0.0, 1.0, 1.5]


# ---- captures with an e4m3 store: what is refused without a device ----

def config(**kw):
    from graph_replay_gb300 import make_config
    base = dict(n_layers=2, d_model=128, n_heads=4, n_kv_heads=2, head_dim=64, ffn_hidden=256, vocab=512, weight_dtype="bf16",
                kv_dtype="e4m3")
    base.update(kw)
    return make_config(**base)


@pytest.mark.parametrize("kw, code, word", [(dict(head_dim=32), 2, "e4m3"), (dict(weight_dtype="e4m3"), 1, "weight_dtype"), (dict(kv_dtype=3), 1, "kv_dtype")])
def test_store_types(B, kw, code, word):
    h = ctypes.c_void_p()
    assert B.lib().dec_init(ctypes.byref(config(**kw)), ctypes.byref(h)) == code and word in B.last_error(None)


def test_store_size(B):
    cap, rows = 8192, 4
    one, two = (B.dec_workspace_size(config(kv_dtype=t), cap, rows, B.DEC_KV_CONTIGUOUS) for t in ("e4m3", "bf16"))
    values = 2 * 2 * rows * 2 * cap * 64          # K and V, layers, rows, heads, positions, dims
    assert 0.85 * values <= two - one <= values   # a byte less a value; the scales and the attention's scratch come on top
    with pytest.raises(B.DecError):
        B.dec_workspace_size(config(), 8200, 1, B.DEC_KV_CONTIGUOUS)     # not a multiple of 16
    with pytest.raises(B.DecError):
        B.dec_workspace_size(config(), 64, 1, B.DEC_KV_PAGED, 8, 64)


@pytest.mark.parametrize("cap,block", [(100, 64), (64, 0), (0, 64), (63, 64)])
def test_empty_caches_of_odd_capacity(B, cap, block):
    from graph_replay_gb300 import KV8Cache
    with pytest.raises(ValueError, match="cap"):   # before anything is allocated: no device is needed
        KV8Cache.empty(1, cap, 1, 64, scale_block=block)


def test_windows_beyond_32_bits(B):
    for window, sinks in ((2 ** 32 + 5, 0), (5, 2 ** 31), (-2 ** 32, 0)):
        with pytest.raises(ValueError, match="32 bits"):
            B.dec_set_window(None, window, sinks)   # before the handle is looked at


def test_growing_a_block_gives_these_values():
    """The exact values behind test_growing_a_block_rounds_its_earlier_tokens."""
    s = R.Store(1, 1, 16, 64, 16)
    one = torch.ones(1, 1, 64, dtype=torch.float64)
    s.append([0], 0, one * 1.125)                    # 448 * 2^-8 >= 1.125: stored as 288 * 2^-8
    assert int(s.e[0, 0, 0]) == -8 and bool((s.x[0, 0, 0] == 288).all())
    s.append([0], 1, one * 1000.0)                   # 1000 * 2^-2 = 250: between 240 and 256, and 288 * 2^-10 between 0.28125
    assert int(s.e[0, 0, 0]) == 2 and bool((s.x[0, 0, 1] == 256).all()) and bool((s.x[0, 0, 0] == 0.28125).all())
    s.append([0], 2, one * 2.0 ** 18)                # 2^18 <= 448 * 2^10: 1.125 * 2^-10 is over half of the least step, 2^-9
    assert int(s.e[0, 0, 0]) == 10 and bool((s.x[0, 0, 2] == 256).all())
    assert bool((s.x[0, 0, 0] == 2.0 ** -9).all()) and bool((s.x[0, 0, 1] == 1.0).all())   # 1024 * 2^-10
    s.append([0], 3, one * 2.0 ** 19)                # half of the least step, to the even one: 0
    assert int(s.e[0, 0, 0]) == 11 and bool((s.x[0, 0, 0] == 0.0).all())
