"""Attention of several new tokens where it can go wrong: what a row may not see, logits that rise, spike or lie far
apart, scales of 0, pages that are none, lengths out of range, graphs, streams and buffers of the caller's."""
import numpy as np
import pytest
import torch

from tests.test_gpu_canary import Guarded
from tests.test_gpu_extend import cache_of, check_extend, ints

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "int8": torch.int8, "fp8": torch.float8_e4m3fn}
FORMS = [("int8", torch.bfloat16, 128, 64, 64), ("fp8", torch.float16, 64, 32, 16), ("int8", torch.float16, 64, 16, 0),
         ("fp8", torch.bfloat16, 128, 64, 0), ("fp16", torch.float16, 128, 64, 0), ("bf16", torch.bfloat16, 64, 48, 0), ("fp8", torch.bfloat16, 128, 64, 32)]
FEW, ONE, MANY = (4, 4), (40, 4), (150, 4)      # (T, query heads over 2 kv heads): 8, 80 (one tile) and 300 rows a kv head


def _sg():
    import bit_trainable_attention_sage_gb300 as sg
    return sg


def appended(kind, d, page, block, K, V):
    """A cache with K, V (B,H,n,d) appended, and the float64 values that it stands for."""
    sg = _sg()
    B, H, n, _ = K.shape
    cache = sg.make_kv_cache(B, H, d, n + 5, dtype=DT[kind], page=page, block=block)
    sg.sage_kv_append(cache, K, V, ints([0] * B))
    return cache, *values_of(cache, n)


def values_of(cache, n):
    out = []
    slots = torch.arange(n)
    for pool, scale in ((cache.K, cache.sK), (cache.V, cache.sV)):
        x = pool.cpu().double()
        if scale is not None:
            x = x * scale.cpu().double().repeat_interleave(cache.block or 1, -1).unsqueeze(-1)
        table = cache.table.cpu().long()
        out.append([x[table[b, slots // cache.page], :, slots % cache.page].permute(1, 0, 2).numpy() for b in range(cache.B)])
    return out


def both(T, Hq):
    return Hq // 2 * T <= 32


@pytest.mark.parametrize("kind,dtype,d,page,block", FORMS)
@pytest.mark.parametrize("T,Hq", [FEW, ONE, MANY])
@pytest.mark.parametrize("shape", ["rising", "falling", "steps", "spikes", "flat", "far below"])
def test_logits(kind, dtype, d, page, block, T, Hq, shape):
    """The running reference where it has to follow, where it must not, and where all logits are alike."""
    sg = _sg()
    g = torch.Generator().manual_seed(d + T)
    n0, B, H = 700, 2, 2
    n = n0 + T
    t = torch.arange(n, dtype=torch.float64) / n
    level = {"rising": t * 60, "falling": -t * 60, "steps": (t * 9).floor() * 25 - 100, "spikes": torch.where(torch.arange(n) % 97 == 41, 40.0 + 30 * t, 0.0),
             "flat": t * 0, "far below": torch.where(torch.arange(n) == 3, 0.0, -25.0)}[shape]
    # q . k / sqrt(d) is `level` and a little more: channel 0 carries it
    K = torch.randn((B, H, n, d), generator=g) * (0.0 if shape == "flat" else 0.05)
    K[..., 0] = (level * d ** 0.5 / 4).float()
    V = torch.randn((B, H, n, d), generator=g)
    Q = torch.randn((B, Hq, T, d), generator=g) * 0.5
    Q[..., 0] = 4.0
    # scales of V that change from block to block
    V *= torch.exp2((torch.arange(n) // 64 % 7 - 3).float()).view(1, 1, n, 1)
    K, V, Q = K.to(dtype).cuda(), V.to(dtype).cuda(), Q.to(dtype).cuda()
    cache, Kd, Vd = appended(kind, d, page, block, K, V)
    O, L = sg.sage_attn_extend(Q, cache, ints([n0] * B))
    assert sg.sage_device_status() == 0
    check_extend(Q, O, L, [n0] * B, [T] * B, Kd, Vd, H, both(T, Hq))


@pytest.mark.parametrize("kind,dtype,d,page,block", FORMS)
@pytest.mark.parametrize("T,Hq", [FEW, ONE, MANY])
def test_hidden_rows_do_not_reach(kind, dtype, d, page, block, T, Hq):
    """A NaN or an infinity in the K, V or scale of a new token reaches that token and those behind it (with scales of
    blocks: those that see any of its block), and no row before."""
    sg = _sg()
    B, H, n0 = 2, 2, 100
    start, t0 = [n0, 0], T // 2
    cache, K, V = cache_of(kind, B, H, d, page, block, [n0 + T, T], seed=T, garbage=False)
    Q = torch.randn(B, Hq, T, d).to(dtype).cuda()
    good_O, good_L = sg.sage_attn_extend(Q, cache, ints(start))
    for what in ("K", "V"):
        for value in (float("nan"), float("inf")):
            saved = [None if x is None else x.clone() for x in (cache.K, cache.V, cache.sK, cache.sV)]
            first = []
            for b in range(B):
                s = start[b] + t0
                p, off = int(cache.table[b, s // page]), s % page
                pool, scale = (cache.K, cache.sK) if what == "K" else (cache.V, cache.sV)
                first.append(t0)
                if scale is not None:
                    scale[p, 1, off // (block or 1)] = value
                    if block:
                        first[b] = max(0, s // block * block - start[b])
                else:
                    pool[p, 1, off, 3] = value
            O, L = sg.sage_attn_extend(Q, cache, ints(start))
            G = Hq // 2
            for b in range(B):
                t1 = first[b]
                assert torch.equal(O[b, :G], good_O[b, :G]) and torch.equal(L[b, :G], good_L[b, :G])          # the other kv head
                if block and b == 1 and t1 == 0:
                    assert not O[b, G:].isfinite().any(-1).all(-1).any() or T == 0
                else:
                    assert torch.allclose(O[b, G:, :t1].float(), good_O[b, G:, :t1].float(), rtol=2.0 ** -6, atol=1e-3), (what, value, b)
                    assert torch.allclose(L[b, G:, :t1], good_L[b, G:, :t1], rtol=1e-5, atol=1e-4)
                if what == "K":
                    if value != value:
                        assert O[b, G:, t0:].isnan().all() and L[b, G:, t0:].isnan().all()
                else:
                    reached = O[b, G:, t0:] if cache.sK is not None else O[b, G:, t0:, 3]
                    assert not reached.isfinite().any(), (what, value, b)
                    if cache.sK is None:
                        rest = torch.arange(d, device="cuda") != 3
                        assert O[b, G:, t0:][..., rest].isfinite().all()
            for x, y in zip((cache.K, cache.V, cache.sK, cache.sV), saved):
                if x is not None:
                    x.view(torch.int8).copy_(y.view(torch.int8))
    assert sg.sage_device_status() == 0


@pytest.mark.parametrize("T,Hq", [FEW, ONE, MANY])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_nan_codes_in_hidden_values(T, Hq, dtype):
    """An E4M3 pool can hold NaN codes under a finite scale."""
    sg = _sg()
    cache, K, V = cache_of("fp8", 1, 2, 64, 32, 32, [60 + T], seed=1, garbage=False)
    Q = torch.randn(1, Hq, T, 64).to(dtype).cuda()
    good = sg.sage_attn_extend(Q, cache, ints([60]))[0]
    s = 60 + T // 2
    cache.V.view(torch.int8)[int(cache.table[0, s // 32]), 0, s % 32, 7] = 0x7F
    O, L = sg.sage_attn_extend(Q, cache, ints([60]))
    G = Hq // 2
    assert O[:, :G, T // 2:, 7].isnan().all() and L.isfinite().all()
    O[:, :G, T // 2:, 7] = good[:, :G, T // 2:, 7]
    assert torch.equal(O, good)


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("block", [0, 16])
@pytest.mark.parametrize("T,Hq", [FEW, ONE, MANY])
def test_scales_of_zero_and_far_apart(kind, block, T, Hq):
    """Blocks of zeros keep their weight in the sum; values 2^40 apart."""
    sg = _sg()
    B, H, d, n0 = 1, 2, 64, 300
    n = n0 + T
    K, V = torch.randn(B, H, n, d), torch.randn(B, H, n, d)
    K[:, :, 32:48] = 0
    V[:, :, 64:112] = 0
    V[:, 0, 200:] *= 2.0 ** -20
    V[:, 0, :50] *= 2.0 ** 20
    Q = torch.randn(B, Hq, T, d).bfloat16().cuda()
    cache, Kd, Vd = appended(kind, d, 16, block, K.bfloat16().cuda(), V.bfloat16().cuda())
    O, L = sg.sage_attn_extend(Q, cache, ints([n0]))
    check_extend(Q, O, L, [n0], [T], Kd, Vd, H, both(T, Hq))


@pytest.mark.parametrize("T,Hq", [FEW, ONE, MANY])
@pytest.mark.parametrize("kind,dtype,d,page,block", FORMS[:1] + FORMS[2:3] + FORMS[4:5])
def test_pages_that_are_none(kind, dtype, d, page, block, T, Hq):
    """Their slots do not exist; reported."""
    sg = _sg()
    n0 = 3 * page + 5
    cache, K, V = cache_of(kind, 2, 2, d, page, block, [n0 + T] * 2, seed=2)
    cache.table[0, 1], cache.table[1, 0] = -1, cache.pages
    Q = torch.randn(2, Hq, T, d).to(dtype).cuda()
    O, L = sg.sage_attn_extend(Q, cache, ints([n0] * 2))
    assert sg.sage_device_status() == 7 and sg.sage_device_status() == 0
    keep = [np.r_[0:page, 2 * page:n0 + T], np.r_[page:n0 + T]]
    check_extend(Q, O, L, [n0 - page] * 2, [T] * 2, [K[b][:, keep[b]] for b in range(2)], [V[b][:, keep[b]] for b in range(2)], 2, both(T, Hq))


@pytest.mark.parametrize("T,Hq", [FEW, ONE, MANY])
def test_lengths_out_of_range(T, Hq):
    """Held to what exists, and reported."""
    sg = _sg()
    cache, K, V = cache_of("int8", 4, 2, 64, 32, 32, [64 + T + 40] * 4, seed=3)
    cap = cache.capacity
    Q = torch.randn(4, Hq, T, 64).bfloat16().cuda()
    # before the first slot; counts out of range
    O, L = sg.sage_attn_extend(Q, cache, ints([-9, 3, 3, 0]), count=ints([T, -1, T + 7, 1]))
    assert sg.sage_device_status() == 7
    seen = [T, 3, 3 + T, 1]
    check_extend(Q, O, L, [0, 3, 3, 0], [T, 0, T, 1], [x[:, :n] for x, n in zip(K, seen)], [x[:, :n] for x, n in zip(V, seen)], 2, both(T, Hq))
    # past the capacity: finite or empty, and nothing outside is read (the last page is no page of the table)
    O, L = sg.sage_attn_extend(Q, cache, ints([cap - 1, cap, cap + 5, 1 << 30]))
    assert sg.sage_device_status() == 7 and O.isfinite().all()


@pytest.mark.parametrize("kind,dtype,d,page,block", FORMS)
def test_one_token_is_decode(kind, dtype, d, page, block):
    sg = _sg()
    lens = [1, 0, 17, 300, 1000]
    cache, _, _ = cache_of(kind, 5, 2, d, page, block, lens, seed=4)
    Q = torch.randn(5, 8, 1, d).to(dtype).cuda()
    a = sg.sage_attn_decode(Q, cache, ints(lens))
    b = sg.sage_attn_extend(Q, cache, ints([max(0, n - 1) for n in lens]), count=ints([min(1, n) for n in lens]))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and sg.sage_device_status() == 0


@pytest.mark.parametrize("T,Hq", [FEW, ONE, MANY, (64, 2)])
@pytest.mark.parametrize("kind,dtype,d,page,block", [FORMS[0], FORMS[4]])
def test_buffers_of_the_callers(kind, dtype, d, page, block, T, Hq):
    """Outputs and a workspace between guards; inputs and the cache unchanged."""
    from bit_trainable_attention_sage_gb300.binding import lib
    sg = _sg()
    start, count = [900, 0, 33], [T, T, 1]
    cache, K, V = cache_of(kind, 3, 2, d, page, block, [s + c for s, c in zip(start, count)], seed=5)
    Q = torch.randn(3, Hq, T, d).to(dtype).cuda()
    c = cache._struct(Q, "Q")
    need = lib().sage_extend_workspace_bytes(c, Hq, T)
    gO, gL, gW = Guarded(Q.numel() * 2), Guarded(3 * Hq * T * 4), Guarded(max(need, 256))
    s, n = ints(start), ints(count)
    tensors = [t for t in (Q, s, n, cache.K, cache.V, cache.sK, cache.sV, cache.table) if t is not None]
    snaps = [t.view(torch.int8).clone() for t in tensors]
    O, L = gO.view(dtype, Q.shape), gL.view(torch.float32, (3, Hq, T))
    st = lib().sage_attn_extend(c, Hq, T, Q.data_ptr(), s.data_ptr(), n.data_ptr(), gO.ptr, gL.ptr, gW.ptr, need, torch.cuda.current_stream().cuda_stream)
    assert st == 0 and sg.sage_device_status() == 0
    assert gO.intact() and gL.intact() and gW.intact() and all(torch.equal(a.view(torch.int8), b) for a, b in zip(tensors, snaps))
    check_extend(Q, O, L, start, count, K, V, 2, both(T, Hq))
    if need:
        assert lib().sage_attn_extend(c, Hq, T, Q.data_ptr(), s.data_ptr(), n.data_ptr(), gO.ptr, gL.ptr, gW.ptr, need - 1, None) == 6


def test_binding_refuses():
    sg = _sg()
    cache = sg.make_kv_cache(2, 2, 64, 64, block=16)
    Q = torch.zeros(2, 4, 3, 64, dtype=torch.bfloat16, device="cuda")
    s = ints([0, 0])
    for bad, err in (((Q.float(), s), TypeError), ((Q[:1], s), ValueError), ((Q, s.long()), TypeError), ((Q, s[:1]), ValueError),
                     ((Q.transpose(1, 2), s), ValueError), ((Q[..., :32], s), ValueError)):
        with pytest.raises(err):
            sg.sage_attn_extend(bad[0], cache, bad[1])
    with pytest.raises(sg.SageError):
        sg.sage_attn_extend(Q[:, :3].contiguous(), cache, s)
    with pytest.raises(sg.SageError):
        sg.sage_attn_extend(Q[:, :, :0].contiguous(), cache, s)
    with pytest.raises(TypeError):
        sg.sage_attn_extend(Q, cache, s, out=torch.empty_like(Q, dtype=torch.float16))


@pytest.mark.parametrize("T,Hq", [FEW, ONE, MANY])
def test_graphs_share_a_workspace_and_streams_do_not(T, Hq):
    """Two captured calls on one workspace of the caller's, replayed in turn with other lengths; two streams at once."""
    from bit_trainable_attention_sage_gb300.binding import lib
    sg = _sg()
    made = [cache_of("int8", 2, 2, 64, 32, 32, [400 + T, 90 + T], seed=s) for s in (6, 7)]
    Qs = [torch.randn(2, Hq, T, 64).bfloat16().cuda() for _ in range(2)]
    ws = torch.empty(max(256, lib().sage_extend_workspace_bytes(made[0][0]._struct(Qs[0], "Q"), Hq, T)), dtype=torch.uint8, device="cuda")
    start = ints([0, 0])
    graphs, outs = [], []
    for (cache, _, _), Q in zip(made, Qs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(sg.sage_attn_extend(Q, cache, start, workspace=ws))
        graphs.append(g)
    for a, b in ((400, 90), (0, 33), (128, 64)):
        start.copy_(ints([a, b]))
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        for (cache, K, V), Q, (O, L) in zip(made, Qs, outs):
            check_extend(Q, O, L, [a, b], [T, T], [k[:, :s + T] for k, s in zip(K, (a, b))], [v[:, :s + T] for v, s in zip(V, (a, b))], 2, both(T, Hq))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    res = [[sg.sage_attn_extend(Q, cache, start, stream=s) for _ in range(5)] for (cache, _, _), Q, s in zip(made, Qs, streams)]
    torch.cuda.synchronize()
    for r, (O, L) in zip(res, outs):
        assert all(torch.equal(o, O) and torch.equal(l, L) for o, l in r)
    assert sg.sage_device_status() == 0


def test_pool_past_2_31_elements():
    """Rows behind 2^31 elements of the pool, 8-bit and 16-bit."""
    sg = _sg()
    for dtype, block in ((torch.int8, 64), (torch.bfloat16, 0)):
        pages, H, page, d, T = (1 << 31) // (64 * 128 * 2) + 64, 2, 64, 128, 70
        K, V = (torch.zeros(pages, H, page, d, dtype=dtype, device="cuda") for _ in range(2))
        s = (torch.zeros(pages, H, 1, device="cuda"), torch.zeros(pages, H, 1, device="cuda")) if block else (None, None)
        table = torch.arange(pages - 8, pages, dtype=torch.int32, device="cuda").flip(0).view(1, 8).contiguous()
        cache = sg.KvCache(K, V, table, sK=s[0], sV=s[1])
        k, v = (torch.randn(1, H, 400, d).bfloat16().cuda() for _ in range(2))
        sg.sage_kv_append(cache, k, v, ints([0]))
        for Hq, T in ((2, 70), (2, 4), (8, 70)):
            Q = torch.randn(1, Hq, T, d).bfloat16().cuda()
            O, L = sg.sage_attn_extend(Q, cache, ints([400 - T]))
            x = [(p[table[0].long()].cpu().double() * (1 if z is None else z[table[0].long()].cpu().double().unsqueeze(-1))).permute(1, 0, 2, 3).reshape(H, -1, d)[:, :400].numpy()
                 for p, z in ((K, s[0]), (V, s[1]))]
            check_extend(Q, O, L, [400 - T], [T], [x[0]], [x[1]], H, Hq // H * T <= 32)
        del K, V, cache


def test_a_conversation():
    """A prompt in chunks, drafted tokens of which some are taken back, and single tokens, over one cache with scales of
    blocks: every answer against 64 bits over what the cache then holds."""
    sg = _sg()
    B, H, Hq, d, page = 2, 2, 8, 128, 64
    cache = sg.make_kv_cache(B, H, d, 1000, dtype=torch.int8, page=page, block=64)
    lens = [0, 0]
    for T, take in ((300, [300, 217]), (64, [64, 64]), (5, [2, 5]), (1, [1, 1]), (4, [4, 0]), (130, [130, 130])):
        k, v, q = (torch.randn(B, h, T, d).bfloat16().cuda() for h in (H, H, Hq))
        count = [T, T] if T != 300 else take
        sg.sage_kv_append(cache, k, v, ints(lens), count=ints(count))
        O, L = sg.sage_attn_extend(q, cache, ints(lens), count=ints(count))
        Kd, Vd = values_of(cache, max(n + c for n, c in zip(lens, count)))
        check_extend(q, O, L, lens, count, [x[:, :n + c] for x, n, c in zip(Kd, lens, count)], [x[:, :n + c] for x, n, c in zip(Vd, lens, count)], H, Hq // H * T <= 32)
        lens = [n + t for n, t in zip(lens, take)]          # (drafts that are taken back are overwritten)
    assert sg.sage_device_status() == 0


@pytest.mark.parametrize("kind,dtype,d,page,block", [FORMS[0], FORMS[1], FORMS[4]])
@pytest.mark.parametrize("T,start", [(5000, 0), (3001, 1777)])
def test_long_prompts(kind, dtype, d, page, block, T, start):
    """Rows here and there of a long prompt of grouped heads, tiles that end inside a head, against 64 bits on the GPU."""
    sg = _sg()
    H, Hq, n = 2, 10, start + T
    K, V = (torch.randn(1, H, n, d).to(dtype).cuda() for _ in range(2))
    Q = torch.randn(1, Hq, T, d).to(dtype).cuda()
    cache = sg.make_kv_cache(1, H, d, n, dtype=DT[kind], page=page, block=block)
    sg.sage_kv_append(cache, K, V, ints([0]))
    O, L = sg.sage_attn_extend(Q, cache, ints([start]))
    assert sg.sage_device_status() == 0
    Kd, Vd = (torch.from_numpy(x[0]).cuda() for x in values_of(cache, n))
    rows = torch.tensor(sorted({0, 1, 127, 128, 255, 256, 257, T // 2, T - 2, T - 1, 1234, 2999}), device="cuda")
    eps = torch.finfo(dtype).eps / 2
    for h in range(Hq):
        s = Q[0, h, rows].double() @ Kd[h // 5].T / d ** 0.5
        s.masked_fill_(torch.arange(n, device="cuda") > start + rows.unsqueeze(1), float("-inf"))
        p = s.softmax(-1)
        want, pv = p @ Vd[h // 5], p @ Vd[h // 5].abs()
        # half a step for the probabilities, half for the output; logits and sums as in check_extend, below 2^-9 here; fp16: what
        # falls below 2^-36 of the largest weight
        bound = (eps + 2.0 ** -9) * pv + eps * want.abs() + n * 2.0 ** -36 * 2.0 ** 9 * Vd.abs().max() + 2.0 ** -25
        assert bool(((O[0, h, rows].double() - want).abs() <= bound).all()), h
        assert bool(((L[0, h, rows].double() - s.logsumexp(-1)).abs() <= 1e-4).all()), h


@pytest.mark.parametrize("B,T,Hq", [(300, 2, 4), (180, 40, 2), (3, 3, 140), (2, 1, 66)])
def test_many_sequences_and_heads(B, T, Hq):
    sg = _sg()
    start = [(37 * b) % 200 for b in range(B)]
    count = [T if b % 3 else max(0, T - 1) for b in range(B)]
    cache, K, V = cache_of("int8", B, 2, 64, 32, 32, [s + c for s, c in zip(start, count)], seed=8)
    Q = torch.randn(B, Hq, T, 64).bfloat16().cuda()
    out, lse = torch.full_like(Q, 7.0), torch.full((B, Hq, T), 7.0, device="cuda")
    O, L = sg.sage_attn_extend(Q, cache, ints(start), count=ints(count), out=out, lse=lse)
    assert O is out and L is lse and sg.sage_device_status() == 0
    check_extend(Q, O, L, start, count, K, V, 2, both(T, Hq))
