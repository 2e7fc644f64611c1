"""Argument checks of the block-scaled cache, before any launch (CPU only: fake device addresses are
never dereferenced)."""
import ctypes

import pytest
import torch

from tests.test_serving_args import _append, _decode, _evict, _kv, sg  # noqa: F401
from tests.test_serving_objects import _pool


@pytest.mark.parametrize("kind,page,status", [
    (1 | 16 << 8, 48, 0), (2 | 32 << 8, 64, 0), (1 | 64 << 8, 64, 0), (16 << 8, 48, 2), (1 | 8 << 8, 64, 2), (1 | 128 << 8, 128, 2),
    (1 | 64 << 8, 96, 2), (2 | 32 << 8, 48, 2), (3 | 16 << 8, 48, 2), (-1, 48, 2), (-(1 << 31), 48, 2), (1 | 24 << 8, 48, 2)])
def test_kinds(sg, kind, page, status):  # noqa: F811
    """Accepted kinds have a workspace size and fail by what else is wrong; the others are refused."""
    c = _kv(sg, kind=kind, page=page, score=None, pos=None)
    assert _append(sg, c, K=None) == (1 if status == 0 else 2)
    assert _decode(sg, c, Q=None) == (1 if status == 0 else 2)
    assert _evict(sg, c) == 2
    big = _kv(sg, kind=kind, page=page, score=None, pos=None, max_pages=10000)
    assert (sg.lib().sage_decode_workspace_bytes(ctypes.byref(big), 6, 0) > 0) == (status == 0)


def test_no_scores(sg):  # noqa: F811
    for kw in (dict(), dict(score=None), dict(pos=None)):
        c = _kv(sg, kind=1 | 16 << 8, **kw)
        assert _append(sg, c) == 2 and _decode(sg, c) == 2 and _evict(sg, c) == 2
    c = _kv(sg, kind=1 | 16 << 8, score=None, pos=None)
    assert _decode(sg, c, score=1) == 1
    assert _append(sg, _kv(sg, kind=1 | 16 << 8, score=None, pos=None, sK=None)) == 1
    assert _append(sg, _kv(sg, kind=1 | 16 << 8, score=None, pos=None, sV=_fake_odd())) == 3


def _fake_odd():
    return 0x10000 * 77 + 8


@pytest.mark.parametrize("kw,what", [
    (dict(block=8), "block must be"), (dict(block=64, page=96), "block must be"), (dict(block=128, page=128), "block must be"),
    (dict(block=-16), "block must be"), (dict(block=16, dtype=torch.float16), "block belongs"), (dict(block=16, score=True), "block belongs")])
def test_make_refuses(sg, kw, what):  # noqa: F811
    v = dict(B=1, H=2, d=64, capacity=100, page=64)
    v.update(kw)
    with pytest.raises(ValueError, match=what):
        sg.make_kv_cache(**v, device="cpu")


@pytest.mark.parametrize("per_page", [3, 8, 32])
def test_cache_refuses_other_blocks(sg, per_page):  # noqa: F811
    K = _pool(page=64)
    s = torch.empty(1).expand(4, 2, per_page)
    with pytest.raises(ValueError, match="block must be"):
        sg.KvCache(K, K, torch.empty(1, dtype=torch.int32).expand(1, 4), sK=s, sV=s)
