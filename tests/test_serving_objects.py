"""The objects of the position and cache calls, on the CPU: what their constructors refuse, and copies of them."""
import pytest
import torch


@pytest.fixture(scope="module")
def sg():
    from bit_trainable_attention_sage_gb300 import build
    build.build()
    import bit_trainable_attention_sage_gb300 as sg
    return sg


def _pool(pages=4, H=2, page=16, d=64):
    return torch.empty(1, dtype=torch.half).expand(pages, H, page, d)


@pytest.mark.parametrize("shape,table,what", [
    (dict(page=24), (1, 4), "multiple of 16"), (dict(page=8), (1, 4), "multiple of 16"), (dict(d=96), (1, 4), "d must be"),
    (dict(H=0), (1, 4), "none may be 0"), (dict(pages=0), (1, 4), "none may be 0"), (dict(), (0, 4), "none may be 0"), (dict(), (1, 0), "none may be 0"),
    (dict(H=8), (8192, 1), "65535"), (dict(page=1 << 24), (1, 64), "2\\^30"),
])
def test_cache_sizes_are_checked_when_it_is_made(sg, shape, table, what):
    """Not first by a call that finds no workspace size for them."""
    K = _pool(**shape)
    with pytest.raises(ValueError, match=what):
        sg.KvCache(K, K, torch.empty(1, dtype=torch.int32).expand(table))


@pytest.mark.parametrize("kw,what", [
    (dict(page=24), "multiple of 16"), (dict(page=0), "none may be 0"), (dict(d=96), "d must be"), (dict(B=0), "none may be 0"),
    (dict(H=0), "none may be 0"), (dict(B=8192, H=8), "65535"), (dict(capacity=1 << 30), "2\\^30"),
])
def test_make_kv_cache_checks_before_it_allocates(sg, kw, what):
    v = dict(B=1, H=2, d=64, capacity=100, page=16)
    v.update(kw)
    with pytest.raises(ValueError, match=what):
        sg.make_kv_cache(**v, device="cpu")


def test_rope_can_be_copied_and_pickled(sg):
    """A Rope held by a module is copied with it, after calls too."""
    import copy
    import pickle
    r = sg.make_rope(128, (16, 24, 24), interleaved=True)
    for _ in range(2):
        for c in (copy.copy(r), copy.deepcopy(r), pickle.loads(pickle.dumps(r)), copy.deepcopy({"rope": r})["rope"]):
            assert (c.d, c.sections, c.freqs, c.interleaved, c.axes, c.rotary) == (r.d, r.sections, r.freqs, True, 3, 128)
            assert list(c._freq) == list(r.freqs) and c._sections is not r._sections and c._made is not r._made
        r._struct(2, 4, 2, 3, torch.float16, 1, False)     # what a call leaves behind
