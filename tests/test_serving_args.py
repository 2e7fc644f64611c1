"""Argument checks of the position and cache calls, before any launch (CPU only: fake device
addresses are never dereferenced)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def sg():
    from bit_trainable_attention_sage_gb300 import build
    build.build()
    import bit_trainable_attention_sage_gb300 as sg
    return sg


def _fake(i):
    return 0x10000 * (i + 1)


def _rope_params(sg, **kw):
    from bit_trainable_attention_sage_gb300.serving import SageRopeParams
    v = dict(B=2, H=4, Hk=2, N=3, d=64, dtype=0, axes=2, pos_batch=2, rotary=32, interleaved=0, inverse=0,
             sections=(ctypes.c_int * 2)(10, 6), freq=(ctypes.c_double * 16)(*[1.0] * 16))
    v.update(kw)
    return SageRopeParams(**v)


@pytest.mark.parametrize("field,value,status", [
    ("B", 0, 1), ("H", 0, 1), ("Hk", -1, 1), ("N", 0, 1), ("d", 96, 2), ("dtype", 3, 2), ("axes", 0, 1), ("axes", 9, 1),
    ("pos_batch", 3, 1), ("rotary", 24, 1), ("rotary", 80, 1), ("rotary", 48, 1), ("interleaved", 2, 1), ("inverse", -1, 1),
    ("sections", (ctypes.c_int * 2)(10, 7), 1), ("sections", (ctypes.c_int * 2)(-1, 17), 1), ("sections", None, 1),
    ("freq", None, 1), ("freq", (ctypes.c_double * 16)(*[float("nan")] * 16), 1),
    ("freq", (ctypes.c_double * 16)(*[float("inf")] * 16), 1),
])
def test_rope_bad_params(sg, field, value, status):
    p = _rope_params(sg, **{field: value})
    f = [_fake(i) for i in range(5)]
    assert sg.lib().sage_rope(ctypes.byref(p), *f, None) == status


def test_rope_bad_pointers(sg):
    p = _rope_params(sg)
    for i in range(5):
        f = [_fake(i) for i in range(5)]
        f[i] = None
        assert sg.lib().sage_rope(ctypes.byref(p), *f, None) == 1
        f[i] = _fake(i) + (2 if i == 2 else 8)
        assert sg.lib().sage_rope(ctypes.byref(p), *f, None) == 3
    assert sg.lib().sage_rope(None, *[_fake(i) for i in range(5)], None) == 1


@pytest.mark.parametrize("kw", [
    dict(d=96, sections=(8,)), dict(d=64, sections=()), dict(d=64, sections=(7,)), dict(d=64, sections=(40,)),
    dict(d=64, sections=(-8, 16)), dict(d=64, sections=(8,), base=0.0), dict(d=64, sections=(8,), base=float("nan")),
    dict(d=64, sections=(8,), freqs=[1.0] * 7), dict(d=64, sections=(8,), freqs=[float("nan")] * 8), dict(d=64, sections=(1,) * 9),
])
def test_make_rope_refuses(sg, kw):
    with pytest.raises(ValueError):
        sg.make_rope(**kw)


def test_make_rope_frequencies(sg):
    r = sg.make_rope(128, (16, 24, 24))
    assert r.rotary == 128 and r.axes == 3 and len(r.freqs) == 64
    assert r.freqs[0] == 1.0 and abs(r.freqs[32] - 1e-2) < 1e-17


def test_rope_binding_refuses(sg):
    r = sg.make_rope(64, (8,))
    pos = torch.zeros(1, 1, 4, dtype=torch.int32)
    with pytest.raises(ValueError):                       # CPU tensors
        sg.sage_rope(torch.zeros(1, 1, 4, 64), None, pos, r)
    with pytest.raises(TypeError):
        sg.sage_rope(torch.zeros(1, 1, 4, 64, dtype=torch.float64), None, pos, r)
    with pytest.raises(ValueError):
        sg.sage_attention(*[torch.zeros(1, 1, 64, 64)] * 3, rope=r)
    with pytest.raises(ValueError):
        sg.sage_attention(*[torch.zeros(1, 1, 64, 64)] * 3, rope=r, positions=pos, qk_norm=True, gamma_q=torch.ones(64))


# ---- cache ----------------------------------------------------------------------------------


def _kv(sg, **kw):
    from bit_trainable_attention_sage_gb300.serving import SageKv
    v = dict(B=2, H=3, d=64, dtype=0, kind=1, page=16, pages=10, max_pages=4, K=_fake(40), V=_fake(41), sK=_fake(42), sV=_fake(43),
             table=_fake(44), score=_fake(45), pos=_fake(46))
    v.update(kw)
    return SageKv(**v)


def _append(sg, c, **kw):
    v = dict(K=_fake(0), V=_fake(1), T=3, start=_fake(2), count=None, mu=None, pos=None)
    v.update(kw)
    return sg.lib().sage_kv_append(None if c is None else ctypes.byref(c), v["K"], v["V"], v["T"], v["start"], v["count"], v["mu"], v["pos"], None)


def _decode(sg, c, **kw):
    v = dict(Hq=6, Q=_fake(0), lens=_fake(1), O=_fake(2), L=_fake(3), score=0, ws=_fake(4), n=1 << 40)
    v.update(kw)
    return sg.lib().sage_attn_decode(None if c is None else ctypes.byref(c), v["Hq"], v["Q"], v["lens"], v["O"], v["L"], v["score"], v["ws"], v["n"], None)


def _evict(sg, c, **kw):
    v = dict(lens=_fake(0), seen=_fake(1), budget=8, recent=2, out=_fake(2), ws=_fake(3), n=1 << 40)
    v.update(kw)
    return sg.lib().sage_kv_evict(None if c is None else ctypes.byref(c), v["lens"], v["seen"], v["budget"], v["recent"], v["out"], v["ws"], v["n"], None)


@pytest.mark.parametrize("fields,status", [
    (dict(B=0), 1), (dict(H=0), 1), (dict(page=0), 1), (dict(pages=0), 1), (dict(max_pages=0), 1), (dict(d=0), 1),
    (dict(dtype=2), 2), (dict(kind=3), 2), (dict(kind=-1), 2), (dict(d=96), 2), (dict(page=24), 2), (dict(max_pages=1 << 26), 2),
    (dict(B=70000), 2), (dict(K=None), 1), (dict(V=None), 1), (dict(table=None), 1), (dict(sK=None), 1), (dict(sV=None), 1),
    (dict(kind=0), 1), (dict(K=_fake(40) + 8), 3), (dict(V=_fake(41) + 2), 3), (dict(table=_fake(44) + 2), 3), (dict(sK=_fake(42) + 4), 3),
    (dict(score=_fake(45) + 4), 3), (dict(pos=_fake(46) + 4), 3),
])
def test_cache_bad_struct(sg, fields, status):
    c = _kv(sg, **fields)
    assert _append(sg, c) == status and _decode(sg, c) == status and _evict(sg, c) == status


def test_cache_calls_refuse(sg):
    c = _kv(sg)
    assert _append(sg, None) == 1 and _decode(sg, None) == 1 and _evict(sg, None) == 1
    for kw, st in ((dict(K=None), 1), (dict(V=None), 1), (dict(start=None), 1), (dict(T=0), 1), (dict(T=-1), 1), (dict(T=1 << 30), 2),
                   (dict(K=_fake(0) + 4), 3), (dict(mu=_fake(9) + 4), 3), (dict(start=_fake(9) + 1), 3), (dict(count=_fake(9) + 2), 3)):
        assert _append(sg, c, **kw) == st, kw
    assert _append(sg, _kv(sg, kind=0, sK=None, sV=None), mu=_fake(9)) == 2      # smoothing a 16-bit cache
    for kw, st in ((dict(Hq=0), 1), (dict(Hq=7), 1), (dict(score=2), 1), (dict(Q=None), 1), (dict(lens=None), 1), (dict(O=None), 1),
                   (dict(L=None), 1), (dict(Q=_fake(0) + 8), 3), (dict(O=_fake(0) + 2), 3), (dict(O=_fake(0)), 1), (dict(Hq=3 << 23), 2)):
        assert _decode(sg, c, **kw) == st, kw
    for kw, st in ((dict(ws=None), 6), (dict(n=100), 6), (dict(ws=_fake(4) + 16), 3)):
        assert _decode(sg, _kv(sg, max_pages=5000), **kw) == st, kw
        assert _decode(sg, c, score=1, **kw) == st, kw
    assert _decode(sg, _kv(sg, score=None), score=1) == 1
    for kw, st in ((dict(lens=None), 1), (dict(seen=None), 1), (dict(out=None), 1), (dict(out=_fake(0)), 1), (dict(out=_fake(1)), 1), (dict(budget=0), 1),
                   (dict(recent=-1), 1), (dict(recent=9), 1), (dict(ws=None), 6), (dict(n=8), 6), (dict(ws=_fake(3) + 8), 3)):
        assert _evict(sg, c, **kw) == st, kw
    assert _evict(sg, _kv(sg, score=None)) == 1 and _evict(sg, _kv(sg, pos=None)) == 1
    assert "range" in sg.sage_status_string(7)


def test_cache_workspaces(sg):
    """Decode: two places a CTA for sums, maxima and sums of exponentials (long caches), and with scores
    a logit a slot and head; evict: at most min(budget, capacity - budget) pairs a row."""
    L = sg.lib()
    c = _kv(sg, B=1, H=1, max_pages=4)
    plain, scored = (L.sage_decode_workspace_bytes(ctypes.byref(c), 4, s) for s in (0, 1))
    assert plain == 0 and scored >= 4 * 64 * 4
    c = _kv(sg, B=1, H=1, max_pages=40000)
    plain, scored = (L.sage_decode_workspace_bytes(ctypes.byref(c), 4, s) for s in (0, 1))
    assert plain >= 456 * 2 * 8 * 66 * 4 and scored >= plain + 4 * 640000 * 4
    assert L.sage_decode_workspace_bytes(ctypes.byref(c), 0, 0) == 0 and L.sage_decode_workspace_bytes(None, 4, 0) == 0
    c = _kv(sg, B=2, H=3, max_pages=4)
    assert L.sage_evict_workspace_bytes(ctypes.byref(c), 8) >= 6 * 2 * 8 * 4
    assert L.sage_evict_workspace_bytes(ctypes.byref(c), 0) == 0
    # big caches do not overflow the sizes
    c = _kv(sg, B=1024, H=8, page=64, max_pages=1 << 14)
    assert L.sage_decode_workspace_bytes(ctypes.byref(c), 32, 1) >= 1024 * 32 * (1 << 20) * 4
    assert L.sage_evict_workspace_bytes(ctypes.byref(c), 1 << 19) >= 2 * 8192 * (1 << 19) * 4


def test_cache_binding_refuses(sg):
    z = torch.zeros
    with pytest.raises(ValueError):                       # CPU tensors
        sg.KvCache(z(4, 2, 16, 64).half(), z(4, 2, 16, 64).half(), z(1, 4, dtype=torch.int32))
    with pytest.raises(ValueError):
        sg.KvCache(z(4, 2, 16, 64), z(4, 2, 16, 64), z(1, 4, dtype=torch.int32))
