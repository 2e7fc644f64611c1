"""Argument checks of sage_attn_extend and of the page calls, before any launch (CPU only: fake device addresses
are never dereferenced)."""
import ctypes

import pytest
import torch

from tests.test_serving_args import _fake, _kv, sg  # noqa: F401


def _extend(sg, c, **kw):  # noqa: F811
    v = dict(Hq=6, T=5, Q=_fake(0), start=_fake(1), count=_fake(2), O=_fake(3), L=_fake(4), ws=_fake(5), n=1 << 40)
    v.update(kw)
    return sg.lib().sage_attn_extend(None if c is None else ctypes.byref(c), v["Hq"], v["T"], v["Q"], v["start"], v["count"], v["O"], v["L"], v["ws"], v["n"], None)


def _call(sg, name, c, **kw):  # noqa: F811
    v = dict(refs=_fake(0), held=_fake(1), a=_fake(2), b=_fake(3), out=_fake(4), ws=_fake(5), n=1 << 40)
    v.update(kw)
    ins = {"sage_kv_resize": [v["a"]], "sage_kv_fork": [v["a"], v["b"]], "sage_kv_compact": []}[name]
    return getattr(sg.lib(), name)(None if c is None else ctypes.byref(c), v["refs"], v["held"], *ins, v["out"], v["ws"], v["n"], None)


def test_extend_refuses(sg):  # noqa: F811
    c = _kv(sg, max_pages=5000)
    assert _extend(sg, None) == 1 and _extend(sg, _kv(sg, d=96)) == 2
    for T in (5, 50):                                     # few rows a kv head, many
        for kw, st in ((dict(Hq=0), 1), (dict(Hq=7), 1), (dict(T=0), 1), (dict(T=-1), 1), (dict(Q=None), 1), (dict(start=None), 1), (dict(O=None), 1),
                       (dict(L=None), 1), (dict(O=_fake(0)), 1), (dict(Q=_fake(0) + 8), 3), (dict(O=_fake(0) + 2), 3), (dict(L=_fake(0) + 4), 3),
                       (dict(start=_fake(1) + 2), 3), (dict(count=_fake(1) + 1), 3), (dict(Hq=3 << 23), 2), (dict(Hq=3 << 10, T=1 << 16), 2),
                       (dict(ws=None), 6), (dict(n=100), 6), (dict(ws=_fake(4) + 16), 3)):
            assert _extend(sg, c, **{"T": T, **kw}) == st, (T, kw)


def test_extend_workspaces(sg):  # noqa: F811
    """Sums of 256 rows, their references and l for each range of slots; none where there are tiles enough."""
    need = lambda c, Hq, T: sg.lib().sage_extend_workspace_bytes(ctypes.byref(c), Hq, T)  # noqa: E731
    long = _kv(sg, B=1, H=1, max_pages=40000)
    assert need(long, 4, 64) >= 16 * 256 * 66 * 4 / 2
    assert need(_kv(sg, B=16, H=3, max_pages=40000), 12, 2048) == 0
    assert need(_kv(sg, B=1, H=1, max_pages=4), 4, 64) == 0               # too short to cut
    assert need(long, 4, 0) == 0 and need(long, 0, 64) == 0 and sg.lib().sage_extend_workspace_bytes(None, 4, 4) == 0
    assert need(long, 4, 3) == sg.lib().sage_decode_workspace_bytes(ctypes.byref(long), 12, 0)


@pytest.mark.parametrize("name", ["sage_kv_resize", "sage_kv_fork", "sage_kv_compact"])
def test_page_calls_refuse(sg, name):  # noqa: F811
    c = _kv(sg, score=None, pos=None)
    assert _call(sg, name, None) == 1 and _call(sg, name, _kv(sg, page=24)) == 2
    cases = [(dict(refs=None), 1), (dict(held=None), 1), (dict(out=None), 1), (dict(refs=_fake(0) + 2), 3), (dict(held=_fake(1) + 1), 3),
             (dict(out=_fake(4) + 2), 3), (dict(ws=None), 6), (dict(n=64), 6), (dict(ws=_fake(5) + 8), 3)]
    if name != "sage_kv_compact":
        cases += [(dict(a=None), 1), (dict(a=_fake(2) + 2), 3), (dict(out=_fake(2)), 1), (dict(out=_fake(1) + 4), 1)]
    if name == "sage_kv_fork":
        cases += [(dict(b=None), 1), (dict(b=_fake(2) + 1), 3), (dict(out=_fake(3) + 4), 1)]
        assert _call(sg, name, _kv(sg, pos=None)) == 2 and _call(sg, name, _kv(sg, score=None)) == 2
    for kw, st in cases:
        assert _call(sg, name, c, **kw) == st, kw


def test_page_workspace(sg):  # noqa: F811
    n = lambda **kw: sg.lib().sage_pages_workspace_bytes(ctypes.byref(_kv(sg, **kw)))  # noqa: E731
    assert n() >= 4 * (3 * 10 + 7 * 2 + 2 + 2 * 4) and n(d=96) == 0 and sg.lib().sage_pages_workspace_bytes(None) == 0
    assert n(B=60000, H=1, max_pages=1 << 20, page=16) >= 4 * 60000 * (1 << 20)


def test_make_refuses(sg):  # noqa: F811
    with pytest.raises(ValueError, match="none may be 0"):
        sg.make_kv_cache(1, 1, 64, 64, pages=0, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        sg.KvCache(torch.zeros(4, 1, 16, 64).half(), torch.zeros(4, 1, 16, 64).half(), torch.zeros(1, 4, dtype=torch.int32),
                   refs=torch.zeros(4, dtype=torch.int32), held=torch.zeros(1, dtype=torch.int32))
