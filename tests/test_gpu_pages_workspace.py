"""The page calls' workspace where the cache's object goes before its calls do."""
import types

import pytest
import torch

from tests.test_gpu_pages import ints, pool

pytestmark = pytest.mark.gpu


def _sg():
    import bit_trainable_attention_sage_gb300 as sg
    return sg


def begun():
    """A pool whose first sequence has 40 slots, its lists, and what stays of the cache when the object goes."""
    sg = _sg()
    cache, model = pool("int8", 3, 2, 64, 16, 20, 5, 16)
    assert sg.sage_kv_resize(cache, ints([40, 0, 17])).tolist() == model.resize([40, 0, 17])
    left = types.SimpleNamespace(**{k: getattr(cache, k) for k in ("K", "V", "sK", "sV", "table", "refs", "held")})
    return cache, model, left


def test_a_call_pending_on_another_stream():
    sg = _sg()
    cache, model, left = begun()
    at, size = cache._pages[2]
    parent, lens = ints([0, 0, 0]), ints([40, 0, 17])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(400_000_000)
    out = sg.sage_kv_fork(cache, parent, lens, stream=s)
    del cache
    others = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(8)]
    pending = not s.query()
    taken = [x for x in others if x.data_ptr() < at + size and at < x.data_ptr() + size]
    s.synchronize()
    assert pending and not taken
    assert out.tolist() == model.fork([0, 0, 0], [40, 0, 17]) and sg.sage_device_status() == 0
    model.check(left)


def test_a_graph_that_outlives_the_cache():
    sg = _sg()
    cache, model, left = begun()
    size = cache._pages[2][1]
    parent, lens = ints([0, 0, 0]), ints([40, 0, 17])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = sg.sage_kv_fork(cache, parent, lens)
        used = sg.sage_kv_compact(cache)
    del cache
    others = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(8)]
    graph.replay()
    torch.cuda.synchronize()
    assert not any(bool(x.any()) for x in others)
    assert out.tolist() == model.fork([0, 0, 0], [40, 0, 17]) and used.tolist() == [model.compact()]
    model.check(left)
    assert sg.sage_device_status() == 0


def test_a_graph_and_calls_beside_it():
    """Replays between other calls of the same cache: each has what it needs in its own workspace."""
    sg = _sg()
    cache, model, left = begun()
    want = ints([50, 20, 17])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        slots = sg.sage_kv_resize(cache, want)
    for w in ([50, 20, 17], [0, 0, 0], [80, 1, 16]):
        want.copy_(ints(w))
        graph.replay()
        assert slots.tolist() == model.resize(w)
        lens = [min(x, 33) for x in w]
        assert sg.sage_kv_fork(cache, ints([0, 2, 1]), ints(lens)).tolist() == model.fork([0, 2, 1], lens)
        model.check(left)
    assert sg.sage_device_status() == 0
