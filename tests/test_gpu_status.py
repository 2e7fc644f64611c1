"""sage_device_status() where two kinds of error are noted at once: the timeout is returned first, the index error
by the next call.

As in test_gpu_timeout.py the timeout is that of the test-only library, whose backward waits for a block that is
never sent and gives up after 0.1 s, in a child process.
"""
import json
import os
import subprocess
import sys
import textwrap

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = textwrap.dedent(r"""
    import ctypes, json, sys
    sys.path.insert(0, ROOT)
    import torch
    import bit_trainable_attention_sage_gb300 as sg
    from bit_trainable_attention_sage_gb300 import build
    fs = ctypes.CDLL(build.build(variant="faultsim"))
    P = ctypes.POINTER(sg.SageParams)
    vp, sz, ci = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    for name in ("sage_quantize_workspace_bytes", "sage_fwd_workspace_bytes", "sage_bwd_workspace_bytes"):
        getattr(fs, name).argtypes = [P]; getattr(fs, name).restype = sz
    fs.sage_quantize_smooth.argtypes = [P] + [vp] * 12 + [sz, vp]
    fs.sage_attn_fwd.argtypes = [P] + [vp] * 12 + [sz, vp]
    fs.sage_attn_bwd.argtypes = [P] + [vp] * 15 + [sz, vp]
    fs.sage_device_status.argtypes = [vp]
    B, H, N, d = 1, 2, 256, 128
    g = torch.Generator().manual_seed(0)
    Q, K, V, dO = (torch.randn((B, H, N, d), generator=g).half().cuda() for _ in range(4))
    p = sg.make_params(B, H, N, d, 0, False)
    st = torch.cuda.current_stream().cuda_stream
    i8 = lambda: torch.empty((B, H, N, d), dtype=torch.int8, device="cuda")
    f32 = lambda *s: torch.empty(s, dtype=torch.float32, device="cuda")
    Qh, Kh, Vh = i8(), i8(), i8()
    sQ, sK, sV = f32(B, H, N // 64), f32(B, H, N // 64), f32(B, H, N // 64)
    muK = f32(B, H, d)
    ws = lambda q: torch.empty(max(q(ctypes.byref(p)), 16), dtype=torch.uint8, device="cuda")
    wq, wf, wb = ws(fs.sage_quantize_workspace_bytes), ws(fs.sage_fwd_workspace_bytes), ws(fs.sage_bwd_workspace_bytes)
    O = torch.empty((B, H, N, d), dtype=torch.float16, device="cuda")
    L = f32(B, H, N)
    dQ, dK, dV = f32(B, H, N, d), f32(B, H, N, d), f32(B, H, N, d)
    ptr = lambda t: None if t is None else t.data_ptr()
    rc = [fs.sage_quantize_smooth(ctypes.byref(p), *map(ptr, (Q, K, V, Qh, Kh, Vh, sQ, sK, sV, muK, None, wq)),
                                  wq.numel(), st)]
    rc.append(fs.sage_attn_fwd(ctypes.byref(p), *map(ptr, (Qh, Kh, Vh, sQ, sK, sV, None, None, None, O, L, wf)),
                               wf.numel(), st))
    fwd_status = fs.sage_device_status(st)
    # an append before the first slot is skipped and noted, then the backward's wait runs out
    from bit_trainable_attention_sage_gb300.serving import SageKv
    fs.sage_kv_append.argtypes = [vp] * 3 + [ci] + [vp] * 5
    pool = torch.zeros((2, 1, 1, 16, 64), dtype=torch.float16, device="cuda")
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    start = torch.full((1,), -5, dtype=torch.int32, device="cuda")
    x = torch.ones((1, 1, 1, 64), dtype=torch.float16, device="cuda")
    kv = SageKv(1, 1, 64, 0, 0, 16, 1, 1, ptr(pool[0]), ptr(pool[1]), None, None, ptr(table), None, None)
    rc.append(fs.sage_kv_append(ctypes.byref(kv), ptr(x), ptr(x), 1, ptr(start), None, None, None, st))
    rc.append(fs.sage_attn_bwd(ctypes.byref(p), *map(ptr, (Qh, Kh, sQ, sK, None, None, None, V, O, L, dO, dQ, dK, dV, wb)),
                               wb.numel(), st))
    both = [fs.sage_device_status(st) for _ in range(3)]
    print(json.dumps(dict(rc=rc, fwd_status=fwd_status, both=both, untouched=bool((pool == 0).all()),
                          after=sg.sage_device_status())))
""").replace("ROOT", repr(ROOT))


def test_a_timeout_does_not_hide_an_index_error():
    r = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0, r.stderr[-2000:]
    out = json.loads(r.stdout.strip().splitlines()[-1])
    assert out["rc"] == [0, 0, 0, 0] and out["fwd_status"] == 0 and out["untouched"]
    assert out["both"] == [5, 7, 0]                   # SAGE_ERR_TIMEOUT, SAGE_ERR_INDEX, SAGE_OK
    assert out["after"] == 0
