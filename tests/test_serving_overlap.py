"""Buffers that the cache calls may not share, refused before any launch (CPU only: fake device addresses are
never dereferenced)."""
import pytest

from tests.test_serving_args import _append, _evict, _fake, _kv, sg  # noqa: F401


@pytest.mark.parametrize("off", [-4, 0, 4])
@pytest.mark.parametrize("which", ["lens", "seen"])
def test_evict_lengths_overlap(sg, which, off):  # noqa: F811
    """lens_out a part of lens or seen: a sequence's new length would be written before another's old one is read."""
    c = _kv(sg)                                            # two sequences: 8 bytes each
    at = _fake(0 if which == "lens" else 1)
    assert _evict(sg, c, out=at + off) == 1
