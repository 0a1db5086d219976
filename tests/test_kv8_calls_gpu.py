"""KV8Cache's own bookkeeping on the GPU: errors of calls on other streams, limits of what it keeps, arguments."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def small(rows=2):
    from graph_replay_gb300 import KV8Cache
    cache = KV8Cache.empty(rows, 64, 2, 64)
    lens = torch.ones(rows, dtype=torch.int32, device="cuda")
    return cache, torch.zeros(rows, 4, 64, device="cuda"), lens


@pytest.mark.parametrize("recorded", [False, True])
def test_check_sees_calls_on_other_streams(recorded):
    """A call that is still to run on a side stream, launched or in a graph, is waited for, and reported once."""
    from graph_replay_gb300 import _binding as B
    cache, q, lens = small()
    bad = torch.tensor([1, 65], dtype=torch.int32, device="cuda")
    out = torch.zeros_like(q)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    if recorded:
        with torch.cuda.graph(graph, stream=side):
            cache.attend(q, bad, out=out)
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(50_000_000)   # some 25 ms
            graph.replay() if recorded else cache.attend(q, bad, out=out)
        with pytest.raises(B.DecError, match="0x2"):
            cache.check()
        cache.check()
    cache.attend(q, lens)
    cache.check()


def test_sizes_kept_are_bounded():
    cache, _, _ = small()
    sizes = [cache.workspace_bytes(n, 4, max_new=n) for n in range(1, 2000)]
    assert len(cache._need) <= 256
    assert sizes[0] == cache.workspace_bytes(1, 4) and sizes[-1] == cache.workspace_bytes(1999, 4, max_new=1999)


@pytest.mark.parametrize("value", [2 ** 31, 2 ** 32 + 5, -2 ** 32])
@pytest.mark.parametrize("name", ["window", "sinks", "max_new"])
def test_numbers_beyond_32_bits_are_refused(name, value):
    cache, q, lens = small()
    kw = dict(window=7) if name == "sinks" else {}
    with pytest.raises(ValueError, match=name):
        cache.attend(q, lens, **kw, **{name: value})
    with pytest.raises(ValueError, match=name):
        cache.workspace_bytes(2, 4, **{name: value})
    if name == "max_new":
        with pytest.raises(ValueError, match=name):
            cache.append(q[:, :2], q[:, 2:], lens, max_new=value)
    cache.attend(q, lens, window=2 ** 31 - 1, sinks=2 ** 31 - 1)   # the largest: no window
    cache.check()
