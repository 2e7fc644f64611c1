"""Guard bytes around every buffer the position and cache calls write, and the ways a program holds
them: outputs and workspaces of its own, threads that share a stream, captured training steps."""
import ctypes
import threading

import pytest
import torch

from tests.cache_common import KINDS, check_decode, filled
from tests.test_gpu_canary import Guarded

pytestmark = pytest.mark.gpu


def _sg():
    import bit_trainable_attention_sage_gb300 as sg
    return sg, sg.lib(), torch.cuda.current_stream().cuda_stream


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype,code,es", [(torch.float16, 0, 2), (torch.float32, 2, 4)])
@pytest.mark.parametrize("N,rotary,inter", [(1, 64, 0), (37, 16, 1), (300, 48, 0)])
def test_rope_stays_inside(dtype, code, es, N, rotary, inter):
    from bit_trainable_attention_sage_gb300.serving import SageRopeParams
    sg, L, st = _sg()
    B, H, Hk, d = 2, 3, 2, 64
    Q, K = torch.randn(B, H, N, d, device="cuda").to(dtype), torch.randn(B, Hk, N, d, device="cuda").to(dtype)
    pos = torch.randint(0, 100, (1, B, N), device="cuda", dtype=torch.int32)
    snaps = Q.clone(), K.clone(), pos.clone()
    out = Guarded(Q.numel() * es), Guarded(K.numel() * es)
    p = SageRopeParams(B, H, Hk, N, d, code, 1, B, rotary, inter, 0, (ctypes.c_int * 1)(rotary // 2),
                       (ctypes.c_double * (rotary // 2))(*[0.5 ** j for j in range(rotary // 2)]))
    assert L.sage_rope(ctypes.byref(p), Q.data_ptr(), K.data_ptr(), pos.data_ptr(), out[0].ptr, out[1].ptr, st) == 0
    torch.cuda.synchronize()
    assert all(g.intact() for g in out) and all(torch.equal(a, b) for a, b in zip((Q, K, pos), snaps))


@pytest.mark.parametrize("kind,d,page,lens,Hq", [
    ("fp16", 64, 16, [33, 0, 16, 47], 4), ("int8", 128, 48, [100, 47, 1], 6), ("fp8", 64, 64, [64, 130], 34),
    ("int8", 64, 32, [5000, 3, 0], 4), ("bf16", 128, 64, [4100, 64], 2), ("fp8", 128, 16, [9000], 32)])
def test_cache_calls_stay_inside(kind, d, page, lens, Hq):
    """Append, decode (with and without scores) and evict on a cache whose every tensor lies between
    guards; what the calls only read is unchanged, pages of no sequence too."""
    sg, L, st = _sg()
    B, H = len(lens), 2
    src, K, V = filled(kind, B, H, d, page, [n + 20 for n in lens], score=True, seed=d + page, garbage=False)
    pages, cap = src.pages, src.capacity
    es = src.K.element_size()
    g = {k: Guarded(t.numel() * t.element_size()) for k in ("K", "V", "sK", "sV", "table", "score", "pos") if (t := getattr(src, k)) is not None}
    as_int = lambda t: t.view({1: torch.int8, 2: torch.int16, 4: torch.int32}[t.element_size()])  # noqa: E731
    for k, buf in g.items():
        t = as_int(getattr(src, k))
        buf.view(t.dtype, t.shape).copy_(t)
    from bit_trainable_attention_sage_gb300.serving import SageKv
    dtype = KINDS[kind] if es == 2 else torch.bfloat16
    c = SageKv(B, H, d, 0 if dtype == torch.float16 else 1, src.kind, page, pages, src.table.shape[1],
               *[g[k].ptr if k in g else None for k in ("K", "V", "sK", "sV", "table", "score", "pos")])
    new = torch.randn(B, H, 20, d, device="cuda").to(dtype)
    before = new.clone()
    assert L.sage_kv_append(ctypes.byref(c), new.data_ptr(), new.data_ptr(), 20, ints(lens).data_ptr(),
                            ints([20 - b for b in range(B)]).data_ptr(), None, None, st) == 0
    Q = torch.randn(B, Hq, 1, d, device="cuda").to(dtype)
    n = ints([x + 20 - b for b, x in enumerate(lens)])
    table = as_int(src.table).clone()
    for score in (0, 1):
        nb = L.sage_decode_workspace_bytes(ctypes.byref(c), Hq, score)
        O, Lse, ws = Guarded(B * Hq * d * 2), Guarded(B * Hq * 4), Guarded(max(nb, 256))
        assert L.sage_attn_decode(ctypes.byref(c), Hq, Q.data_ptr(), n.data_ptr(), O.ptr, Lse.ptr, score, ws.ptr, nb, st) == 0
        torch.cuda.synchronize()
        assert O.intact() and Lse.intact() and ws.intact()
        assert torch.isfinite(O.view(dtype, (B * Hq * d,)).float()).all()
    budget = max(lens) // 2 + 1
    nb = L.sage_evict_workspace_bytes(ctypes.byref(c), budget)
    new_lens, ws = Guarded(4 * B), Guarded(nb)
    seen = ints([10 ** 6] * B)
    assert L.sage_kv_evict(ctypes.byref(c), n.data_ptr(), seen.data_ptr(), budget, 1, new_lens.ptr, ws.ptr, nb, st) == 0
    torch.cuda.synchronize()
    assert new_lens.intact() and ws.intact() and all(b.intact() for b in g.values())
    assert torch.equal(g["table"].view(torch.int32, src.table.shape), table) and torch.equal(new, before)
    assert sg.sage_device_status() == 0
    owned = torch.zeros(pages, dtype=torch.bool)
    for b, x in enumerate(lens):
        owned[table[b, :-(-(x + 20) // page)].long().cpu()] = True
    spare = ~owned
    assert torch.equal(g["K"].view(as_int(src.K).dtype, src.K.shape)[spare.cuda()], as_int(src.K)[spare.cuda()])


def test_outputs_and_workspaces_of_the_caller():
    sg, L, _ = _sg()
    lens = [3000, 5]
    cache, K, V = filled("int8", 2, 1, 64, 64, lens, score=True)
    Q = torch.randn(2, 4, 1, 64, device="cuda").half()
    nb = L.sage_decode_workspace_bytes(cache._struct(Q, "Q"), 4, 1)
    ws, O, Lse = torch.empty(nb, dtype=torch.uint8, device="cuda"), torch.empty_like(Q), torch.empty(2, 4, 1, device="cuda")
    got = sg.sage_attn_decode(Q, cache, ints(lens), score=True, out=O, lse=Lse, workspace=ws)
    assert got[0] is O and got[1] is Lse
    check_decode(Q, O, Lse, lens, K, V, 1)
    with pytest.raises(sg.SageError):
        sg.sage_attn_decode(Q, cache, ints(lens), score=True, workspace=ws[:nb - 512])
    with pytest.raises(sg.SageError):
        sg.sage_attn_decode(Q, cache, ints(lens), out=Q)
    for bad in (dict(out=O.float()), dict(lse=Lse.half()), dict(out=O[:, :2]), dict(workspace=ws.cpu())):
        with pytest.raises((TypeError, ValueError)):
            sg.sage_attn_decode(Q, cache, ints(lens), **bad)
    # a view whose strides are those of a contiguous tensor is taken, a strided one refused
    assert torch.equal(sg.sage_attn_decode(Q.expand(2, 4, 3, 64)[:, :, :1], cache, ints(lens))[0], O)
    with pytest.raises(ValueError):
        sg.sage_attn_decode(torch.randn(2, 4, 3, 64, device="cuda").half()[:, :, :1], cache, ints(lens))
    with pytest.raises(TypeError):
        sg.sage_attn_decode(Q, cache, torch.tensor(lens, device="cuda"))             # int64
    with pytest.raises(ValueError):
        sg.sage_kv_evict(cache, ints(lens), ints(lens), budget=10, recent=11)
    out = ints([0, 0])
    assert sg.sage_kv_evict(cache, ints(lens), ints([10 ** 6] * 2), budget=100, out=out) is out and out.tolist() == [100, 5]


def test_threads_that_share_a_stream():
    """Several host threads call on one cache and one stream: each call's launches and workspace are
    its own."""
    sg, _, _ = _sg()
    lens = [20000, 300]
    cache, K, V = filled("bf16", 2, 2, 64, 64, lens)
    n = ints(lens)
    Qs = [torch.randn(2, 8, 1, 64, device="cuda").bfloat16() for _ in range(8)]
    want = [sg.sage_attn_decode(q, cache, n) for q in Qs]
    torch.cuda.synchronize()
    got = [[] for _ in Qs]

    def work(i):
        for _ in range(20):
            got[i].append(sg.sage_attn_decode(Qs[i], cache, n))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(Qs))]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    for w, outs in zip(want, got):
        assert all(torch.equal(w[0], o) and torch.equal(w[1], l) for o, l in outs)


def test_rotary_step_captured():
    """Forward and backward of sage_rotary captured into a graph (no eager graph of the leaves alive, as
    PyTorch wants it); replays follow the inputs."""
    sg, _, _ = _sg()
    rope = sg.make_rope(64, (16, 16))
    Q, K = (torch.randn(1, 2, 5, 64, device="cuda", requires_grad=True) for _ in range(2))
    pos = torch.randint(0, 50, (2, 1, 5), device="cuda", dtype=torch.int32)
    dQ, dK = torch.randn_like(Q), torch.randn_like(K)

    def step():
        return torch.autograd.grad(sg.sage_rotary(Q, K, pos, rope), (Q, K), (dQ, dK))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads = step()
    pos.add_(7)
    dQ.normal_()
    graph.replay()
    want = sg.sage_rope(dQ, dK, pos, rope, inverse=True)
    assert torch.equal(grads[0], want[0]) and torch.equal(grads[1], want[1])
