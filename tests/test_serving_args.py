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
