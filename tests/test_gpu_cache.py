"""The paged key-value cache: append (codes bit for bit), one-token attention (64-bit reference,
derived tolerances) and eviction (exact), alone and run together."""
import numpy as np
import pytest
import torch

from tests.cache_common import KINDS, check_decode, codes_of, evict64, filled

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def bits(t):
    return t.view(torch.int8) if t.element_size() == 1 else t.view({2: torch.int16, 4: torch.int32}[t.element_size()])


def status(sg):
    return sg.sage_device_status()


# ---- append ---------------------------------------------------------------------------------


def appended(cache_kind, K, V, starts, counts, table, page, pools, scales, mu=None):
    """The pools and scales after an append, on the CPU, from the definition."""
    for which, x in enumerate((K, V)):
        y = x.float()
        if which == 0 and mu is not None:
            y = y - mu.unsqueeze(2)
        if cache_kind in ("int8", "fp8"):
            c, s = codes_of(y, cache_kind)
        else:
            c, s = x, None
        for b, (a, n) in enumerate(zip(starts, counts)):
            for t in range(n):
                p, r = int(table[b, (a + t) // page]), (a + t) % page
                bits(pools[which])[p, :, r] = bits(c)[b, :, t]
                if s is not None:
                    scales[which][p, :, r] = s[b, :, t]


@pytest.mark.parametrize("kind", ["fp16", "bf16", "int8", "fp8"])
@pytest.mark.parametrize("B,H,T,d,page,starts,counts,mu", [
    (3, 2, 1, 128, 16, [0, 15, 16], [1, 0, 1], False),
    (2, 3, 37, 64, 48, [5, 0], [37, 20], True),
    (4, 1, 130, 128, 64, [0, 63, 64, 1], [130, 1, 0, 129], True),
])
def test_append(kind, B, H, T, d, page, starts, counts, mu):
    import bit_trainable_attention_sage_gb300 as sg
    dtype = KINDS[kind] if kind in ("fp16", "bf16") else torch.bfloat16 if T == 37 else torch.float16
    g = torch.Generator().manual_seed(T)
    K, V = torch.randn(B, H, T, d, generator=g).to(dtype), (3 * torch.randn(B, H, T, d, generator=g)).to(dtype)
    K[0, 0, 0] = 0                                  # a zero row: scale 0, codes 0
    mu_t = torch.randn(B, H, d, generator=g) if mu and kind in ("int8", "fp8") else None
    lens = [max(a + T, 1) for a in starts]
    cache, _, _ = filled(kind, B, H, d, page, lens, seed=T, score=True, garbage=False)
    pools = [cache.K.cpu().clone(), cache.V.cpu().clone()]
    scales = [None if cache.sK is None else cache.sK.cpu().clone(), None if cache.sV is None else cache.sV.cpu().clone()]
    score, pos = cache.score.cpu().clone(), cache.pos.cpu().clone()
    pos0 = [100 * b for b in range(B)]
    sg.sage_kv_append(cache, K.cuda(), V.cuda(), ints(starts), count=ints(counts), mu=None if mu_t is None else mu_t.cuda(), pos=ints(pos0))
    appended(kind, K, V, starts, counts, cache.table.cpu(), page, pools, scales, mu_t)
    for b, (a, n) in enumerate(zip(starts, counts)):
        score[b, :, a:a + n] = 0
        pos[b, :, a:a + n] = torch.arange(pos0[b], pos0[b] + n, dtype=torch.int32)
    assert status(sg) == 0
    # everything, what the call had no business with included
    for got, want in zip((cache.K, cache.V, cache.score, cache.pos), pools + [score, pos]):
        assert torch.equal(bits(got.cpu()), bits(want))
    if scales[0] is not None:
        for got, want in zip((cache.sK, cache.sV), scales):
            assert torch.equal(bits(got.cpu()), bits(want))


@pytest.mark.parametrize("kind", ["int8", "fp8"])
def test_append_extreme_rows(kind):
    """Subnormal and tiny rows (scales that round), a single large value, all equal."""
    import bit_trainable_attention_sage_gb300 as sg
    cache, _, _ = filled(kind, 1, 1, 64, 16, [32], garbage=False)
    x = torch.randn(1, 1, 32, 64, generator=torch.Generator().manual_seed(0))
    for i, e in enumerate([0, -30, -60, -100, -120, -126, -130, -133, 60, 100, 120]):
        x[0, 0, i] *= 2.0 ** e
    x[0, 0, 12], x[0, 0, 13] = 1.0, 0.0
    x[0, 0, 13, 5] = -3e38
    K = x.to(torch.bfloat16)
    pools = [cache.K.cpu().clone(), cache.V.cpu().clone()]
    scales = [cache.sK.cpu().clone(), cache.sV.cpu().clone()]
    sg.sage_kv_append(cache, K.cuda(), K.cuda(), ints([0]))
    appended(kind, K, K, [0], [32], cache.table.cpu(), 16, pools, scales)
    assert torch.equal(bits(cache.sK.cpu()), bits(scales[0]))
    assert torch.equal(bits(cache.K.cpu()), bits(pools[0])) and torch.equal(bits(cache.V.cpu()), bits(pools[1]))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("mu", [False, True])
@pytest.mark.parametrize("kind", ["int8", "fp8"])
def test_append_keeps_nan_and_infinity(kind, mu, d):
    """A NaN or infinite value in a row shows in the row's scale (INT8 has no code for it) and so in what is
    read back; all other rows, of the same warp too, keep their bits."""
    import bit_trainable_attention_sage_gb300 as sg
    T = 40
    g = torch.Generator().manual_seed(d)
    K, V = (torch.randn(1, 2, T, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    mu_t = torch.randn(1, 2, d, generator=g).cuda() if mu else None

    def stored(K, V):
        cache = sg.make_kv_cache(1, 2, d, T, dtype=KINDS[kind], page=48)
        sg.sage_kv_append(cache, K, V, ints([0]), mu=mu_t)
        assert status(sg) == 0
        return cache

    clean = stored(K, V)
    K2, V2 = K.clone(), V.clone()
    for i, bad in enumerate((float("nan"), float("inf"), float("-inf"))):
        for c in (0, d // 2 + 3, d - 1):
            K2[0, 0, 3 * c % 13 + i * 13, c] = bad
        V2[0, 1, 5 + i, 9] = bad
    V2[0, 0, 20], V2[0, 0, 20, 1] = 0, float("nan")      # the rest of the row zero
    got = stored(K2, V2)
    for x, x2, pool, pool2, scale, scale2 in ((K, K2, clean.K, got.K, clean.sK, got.sK), (V, V2, clean.V, got.V, clean.sV, got.sV)):
        ok = torch.isfinite(x2).all(-1)[0]
        assert not ok.all()
        nan = torch.isnan(x2).any(-1)[0]
        assert torch.equal(torch.isnan(scale2[0, :, :T]), nan) and torch.equal(torch.isinf(scale2[0, :, :T]), ~ok & ~nan)
        assert torch.equal(bits(scale2[0, :, :T][ok]), bits(scale[0, :, :T][ok]))
        assert torch.equal(bits(pool2[0, :, :T][ok]), bits(pool[0, :, :T][ok]))
    Q = torch.ones(1, 2, 1, d, dtype=torch.bfloat16, device="cuda")
    O, L = sg.sage_attn_decode(Q, got, ints([T]))
    assert torch.isnan(L[0, 0]).all() and torch.isnan(O[0, 0]).all()
    assert torch.isfinite(L[0, 1]).all() and not torch.isfinite(O[0, 1]).any()


def test_append_long_prompt_default_count_and_positions():
    import bit_trainable_attention_sage_gb300 as sg
    T = 1000
    cache = sg.make_kv_cache(2, 4, 128, 1100, dtype=torch.int8, score=True)
    g = torch.Generator().manual_seed(0)
    K, V = (torch.randn(2, 4, T, 128, generator=g).half() for _ in range(2))
    sg.sage_kv_append(cache, K.cuda(), V.cuda(), ints([0, 100]))
    c, s = codes_of(K.float(), "int8")
    t = torch.arange(T)
    for b, a in enumerate((0, 100)):
        p = cache.table.cpu()[b, (a + t) // 64].long()
        assert torch.equal(cache.K.cpu()[p, :, (a + t) % 64], c[b].transpose(0, 1))
        assert torch.equal(cache.sK.cpu()[p, :, (a + t) % 64], s[b].transpose(0, 1))
        assert torch.equal(cache.pos.cpu()[b, 0, a:a + T], (a + t).int())


def test_append_out_of_range_is_skipped_and_reported():
    """Slots past the capacity, negative starts, pages that are none, counts past T: skipped, the
    rest written, SAGE_ERR_INDEX once."""
    import bit_trainable_attention_sage_gb300 as sg
    cache, _, _ = filled("fp16", 3, 1, 64, 16, [48, 48, 48], garbage=False, score=True)
    table = cache.table
    table[:, 3] = ints([10 ** 6, -1, 2 ** 31 - 1])        # the fourth page of each is none
    before = cache.K.clone(), cache.V.clone()
    K = torch.randn(3, 1, 20, 64, device="cuda").half()
    sg.sage_kv_append(cache, K, K, ints([40, 60, -5]), count=ints([20, 30, 3]))
    assert status(sg) == 7 and status(sg) == 0
    want = before[0].clone()
    tb = table.cpu()
    for t in range(8):                                    # sequence 0: slots 40 .. 47 have a page
        want[int(tb[0, (40 + t) // 16]), 0, (40 + t) % 16] = K[0, 0, t]
    assert torch.equal(cache.K, want)                     # 1: slots 60 .. have none; 2: slots -5 .. -3


# ---- decode ---------------------------------------------------------------------------------

SHAPES = [
    # Hq, H, d, page, lens
    (4, 4, 64, 16, [1, 0, 15, 16, 17, 63, 64, 65, 130]),
    (8, 1, 128, 64, [200, 1, 0, 777]),
    (6, 2, 128, 48, [333, 64, 5]),
    (9, 1, 64, 16, [100, 31]),
    (32, 2, 128, 128, [129, 1, 640]),
    (17, 1, 128, 32, [70, 0, 200]),
    (40, 1, 64, 64, [257]),
    (2, 2, 128, 16, [0, 0]),
]


@pytest.mark.parametrize("kind", ["fp16", "bf16", "int8", "fp8"])
@pytest.mark.parametrize("Hq,H,d,page,lens", SHAPES)
@pytest.mark.parametrize("score", [False, True])
def test_decode(kind, Hq, H, d, page, lens, score):
    import bit_trainable_attention_sage_gb300 as sg
    B = len(lens)
    q_dtype = KINDS[kind] if kind in ("fp16", "bf16") else (torch.bfloat16 if d == 128 else torch.float16)
    cache, K, V = filled(kind, B, H, d, page, lens, seed=Hq + d, score=score)
    Q = torch.randn(B, Hq, 1, d, generator=torch.Generator().manual_seed(1)).to(q_dtype).cuda()
    was = cache.score.clone() if score else None
    O, L = sg.sage_attn_decode(Q, cache, ints(lens), score=score)
    assert status(sg) == 0
    assert O.dtype == Q.dtype and O.shape == Q.shape and L.shape == (B, Hq, 1)
    check_decode(Q, O, L, lens, K, V, H, cache.score, was)


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_decode_long_split(kind):
    """A sequence that every CTA shares, beside short ones; peaked logits (one key decides)."""
    import bit_trainable_attention_sage_gb300 as sg
    lens = [3, 33333, 1, 500]
    cache, K, V = filled(kind, 4, 1, 64, 64, lens, seed=5, score=True, v_scale=50.0)
    Q = (4 * torch.randn(4, 5, 1, 64, generator=torch.Generator().manual_seed(1))).to(torch.bfloat16).cuda()
    was = cache.score.clone()
    O, L = sg.sage_attn_decode(Q, cache, ints(lens), score=True)
    check_decode(Q, O, L, lens, K, V, 1, cache.score, was)


def test_decode_many_sequences():
    """More sequences than a CTA has threads, most of them empty or short."""
    import bit_trainable_attention_sage_gb300 as sg
    rng = np.random.default_rng(0)
    lens = [int(n) for n in rng.integers(0, 40, 700)]
    for b in range(0, 700, 50):
        lens[b] = int(rng.integers(100, 300))
    lens[-3:] = [0, 0, 0]
    cache, K, V = filled("fp16", 700, 2, 64, 16, lens, seed=2)
    Q = torch.randn(700, 4, 1, 64, generator=torch.Generator().manual_seed(1)).half().cuda()
    O, L = sg.sage_attn_decode(Q, cache, ints(lens))
    check_decode(Q, O, L, lens, K, V, 2)


@pytest.mark.parametrize("kind", ["int8", "fp8"])
def test_decode_scales_far_apart(kind):
    """V scales that span the range over the tokens, small first: the running power of two moves."""
    import bit_trainable_attention_sage_gb300 as sg
    n = 300
    cache, K, V = filled(kind, 1, 1, 128, 16, [n], seed=9)
    t = torch.arange(n)
    rows = (cache.table.cpu()[0, t // 16].long().cuda(), 0, (t % 16).cuda())
    f = torch.logspace(-20, 3, n, base=10.0)[torch.randperm(n, generator=torch.Generator().manual_seed(0))] if kind == "fp8" \
        else torch.logspace(-20, 3, n, base=10.0)
    f = f.float()
    sv = cache.sV[rows].cpu()
    V = [(V[0] / sv.double().numpy()[None, :, None]) * (sv * f).double().numpy()[None, :, None]]
    cache.sV[rows] = (sv * f).cuda()
    for q_dtype, qs in ((torch.float16, 1.0), (torch.bfloat16, 1e-30), (torch.bfloat16, 3.0), (torch.float16, 6e-8)):
        Q = (qs * torch.randn(1, 3, 1, 128, generator=torch.Generator().manual_seed(1))).to(q_dtype).cuda()
        O, L = sg.sage_attn_decode(Q, cache, ints([n]))
        check_decode(Q, O, L, [n], K, V, 1)


@pytest.mark.parametrize("score", [False, True])
@pytest.mark.parametrize("kind,lens", [
    ("fp16", [40, 100]),                                 # a pair in one cluster
    ("fp8", [9, 30]),
    ("bf16", [20000, 33]),                               # few long sequences: joined a head a block
    ("int8", [20000, 33]),
    ("int8", [300 + 7 * b for b in range(90)]),          # joined where runs meet, and whole pairs
    ("bf16", [300 + 7 * b for b in range(90)]),
])
def test_decode_keeps_a_nan(kind, lens, score):
    """A NaN in one head's q makes that head's O and L NaN (not L = -inf, which says: no slots) and
    leaves every other head's bits as they are; scores of its kv head become NaN, others keep theirs."""
    import bit_trainable_attention_sage_gb300 as sg
    B, d = len(lens), 64
    dtype = KINDS[kind] if kind in ("fp16", "bf16") else torch.float16
    cache, _, _ = filled(kind, B, 2, d, 64, lens, seed=3, score=True)
    was = cache.score.clone()
    Q = torch.randn(B, 6, 1, d, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    O, L = sg.sage_attn_decode(Q, cache, ints(lens), score=score)
    clean = cache.score.clone()
    cache.score.copy_(was)
    Q2 = Q.clone()
    Q2[0, 1, 0, 5] = float("nan")
    O2, L2 = sg.sage_attn_decode(Q2, cache, ints(lens), score=score)
    assert status(sg) == 0
    assert torch.isnan(O2[0, 1]).all() and torch.isnan(L2[0, 1]).all()
    O2[0, 1], L2[0, 1] = O[0, 1], L[0, 1]
    assert torch.equal(bits(O2), bits(O)) and torch.equal(bits(L2), bits(L))
    if score:
        assert torch.isnan(cache.score[0, 0, :lens[0]]).all()
        cache.score[0, 0, :lens[0]] = clean[0, 0, :lens[0]]
        assert torch.equal(bits(cache.score), bits(clean))


@pytest.mark.parametrize("kind", ["fp16", "bf16", "int8", "fp8"])
@pytest.mark.parametrize("n", [50, 5000])
def test_decode_keeps_a_nan_of_the_cache(kind, n):
    """A NaN in a cached V (8 bits: in its scale) reaches O alone; one in a cached K every head's O and L
    of its kv head.  The other kv head's bits stay."""
    import bit_trainable_attention_sage_gb300 as sg
    dtype = KINDS[kind] if kind in ("fp16", "bf16") else torch.float16
    Q = torch.randn(1, 4, 1, 64, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    for which in ("V", "K"):
        cache, _, _ = filled(kind, 1, 2, 64, 16, [n], seed=4)
        O, L = sg.sage_attn_decode(Q, cache, ints([n]))
        t = n // 2
        page = int(cache.table[0, t // 16])
        if kind in ("int8", "fp8"):
            getattr(cache, "s" + which)[page, 0, t % 16] = float("nan")
        else:
            getattr(cache, which)[page, 0, t % 16, 7] = float("nan")
        O2, L2 = sg.sage_attn_decode(Q, cache, ints([n]))
        assert torch.equal(bits(O2[:, 2:]), bits(O[:, 2:])) and torch.equal(bits(L2[:, 2:]), bits(L[:, 2:]))
        if which == "K":
            assert torch.isnan(O2[:, :2]).all() and torch.isnan(L2[:, :2]).all()
        else:
            where = slice(None) if kind in ("int8", "fp8") else slice(7, 8)
            assert torch.isnan(O2[:, :2, :, where]).all() and torch.equal(bits(L2), bits(L))


def test_decode_shared_prefix_pages():
    """Two sequences read the same pages; scores stay each sequence's own."""
    import bit_trainable_attention_sage_gb300 as sg
    cache, K, V = filled("bf16", 3, 2, 64, 16, [80, 90, 40], shared=[(1, 0, 4)], score=True, garbage=False)
    V[1][:, :64], K[1][:, :64] = V[0][:, :64], K[0][:, :64]
    Q = torch.randn(3, 4, 1, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    was = cache.score.clone()
    O, L = sg.sage_attn_decode(Q, cache, ints([80, 90, 40]), score=True)
    check_decode(Q, O, L, [80, 90, 40], K, V, 2, cache.score, was)


def test_decode_far_rows_of_a_large_pool():
    """Rows past 2^31 elements of the pool."""
    import bit_trainable_attention_sage_gb300 as sg
    pages, n = 270000, 100
    small, K, V = filled("int8", 1, 1, 128, 64, [n], spare=0, garbage=False)
    pool = [torch.empty((pages, 1, 64, 128), dtype=torch.int8, device="cuda") for _ in range(2)]
    scale = [torch.empty((pages, 1, 64), device="cuda") for _ in range(2)]
    table = ints([[pages - 1, pages - 2]])
    for i, p in enumerate((pages - 1, pages - 2)):
        src = int(small.table[0, i])
        pool[0][p], pool[1][p], scale[0][p], scale[1][p] = small.K[src], small.V[src], small.sK[src], small.sV[src]
    cache = sg.KvCache(pool[0], pool[1], table, sK=scale[0], sV=scale[1])
    Q = torch.randn(1, 2, 1, 128, generator=torch.Generator().manual_seed(1)).half().cuda()
    O, L = sg.sage_attn_decode(Q, cache, ints([n]))
    check_decode(Q, O, L, [n], K, V, 1)
    x = torch.randn(1, 1, 1, 128, device="cuda").half()
    sg.sage_kv_append(cache, x, x, ints([n]))
    c, s = codes_of(x.cpu().float(), "int8")
    assert torch.equal(pool[0][pages - 2, 0, n - 64].cpu(), c[0, 0, 0]) and scale[1][pages - 2, 0, n - 64].cpu() == s[0, 0, 0]


def test_decode_bad_pages_and_lengths():
    """A page that is none is masked, a length is held to the capacity, and both are reported."""
    import bit_trainable_attention_sage_gb300 as sg
    lens = [100, 40, 64]
    cache, K, V = filled("fp16", 3, 1, 64, 16, lens, garbage=False, score=True)
    table = cache.table
    table[0, 2] = -1
    table[1, :3] = 10 ** 6                               # sequence 1 has no page at all
    Q = torch.randn(3, 2, 1, 64, generator=torch.Generator().manual_seed(1)).half().cuda()
    was = cache.score.clone()
    O, L = sg.sage_attn_decode(Q, cache, ints(lens), score=True)
    assert status(sg) == 7 and status(sg) == 0
    keep = [i for i in range(100) if i // 16 != 2]
    got = cache.score.clone()
    assert torch.equal(got[0, 0, 32:48], was[0, 0, 32:48]) and torch.equal(got[1], was[1])
    check_decode(Q[:1], O[:1], L[:1], [len(keep)], [K[0][:, keep]], [V[0][:, keep]], 1)
    assert torch.all(O[1] == 0) and torch.all(L[1] == float("-inf"))
    check_decode(Q[2:], O[2:], L[2:], [64], [K[2]], [V[2]], 1)
    O2, L2 = sg.sage_attn_decode(Q, cache, ints([-3, 0, 64]))
    assert status(sg) == 7
    assert torch.all(O2[:2] == 0) and torch.equal(O2[2], O[2])


def test_decode_repeats_bit_for_bit_on_streams_and_in_graphs():
    """The same call twice, on another stream, and replayed from two graphs that share a workspace."""
    import bit_trainable_attention_sage_gb300 as sg
    lens = ints([3000, 17, 0, 900])
    cache, K, V = filled("int8", 4, 2, 128, 64, [3000, 17, 0, 900], score=True)
    Q = torch.randn(4, 8, 1, 128, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    s0 = cache.score.clone()
    O, L = sg.sage_attn_decode(Q, cache, lens, score=True)
    s1 = cache.score.clone()
    side = torch.cuda.Stream()
    for stream in (None, side):
        cache.score.copy_(s0)
        torch.cuda.synchronize()
        O2, L2 = sg.sage_attn_decode(Q, cache, lens, score=True, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(O, O2) and torch.equal(L, L2) and torch.equal(s1, cache.score)
    ws = torch.empty(sg.lib().sage_decode_workspace_bytes(cache._struct(Q, "Q"), 8, 1), dtype=torch.uint8, device="cuda")
    lens2 = lens.clone()
    graphs = []
    for x in (lens, lens2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = sg.sage_attn_decode(Q, cache, x, score=True, workspace=ws)
        graphs.append((g, out))
    lens2.copy_(ints([1, 1000, 5, 0]))
    cache.table[1, :16] = cache.table[0, :16]             # sequence 1 now reads sequence 0's pages, 2 has none
    cache.score.copy_(s0)
    O, L = sg.sage_attn_decode(Q, cache, lens, score=True)
    s1 = cache.score.clone()
    cache.score.copy_(s0)
    Ow, Lw = sg.sage_attn_decode(Q, cache, lens2, score=True)
    sw = cache.score.clone()
    cache.score.copy_(s0)
    graphs[1][0].replay()
    torch.cuda.synchronize()
    assert torch.equal(sw, cache.score)
    cache.score.copy_(s0)
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert torch.equal(s1, cache.score)
    assert torch.equal(graphs[0][1][0], O) and torch.equal(graphs[1][1][0], Ow) and torch.equal(graphs[1][1][1], Lw)
    assert status(sg) == 7                                # sequence 2's five slots


# ---- evict ----------------------------------------------------------------------------------


def evicted(cache, lens, seen, budget, recent):
    """Everything after an eviction, on the CPU: by sorting, row by row."""
    out = {k: None if (t := getattr(cache, k)) is None else t.cpu().clone() for k in ("K", "V", "sK", "sV", "score", "pos")}
    table, page = cache.table.cpu().tolist(), cache.page
    score, pos = out["score"].clone(), out["pos"].clone()
    for b, n in enumerate(lens):
        for h in range(cache.H):
            dst, src = evict64(score[b, h].tolist(), pos[b, h].tolist(), n, seen[b], budget, recent)
            assert len(dst) == len(src)
            for d, s in zip(dst, src):
                for k in ("K", "V", "sK", "sV"):
                    if out[k] is not None:
                        x = bits(out[k])
                        x[table[b][d // page], h, d % page] = x[table[b][s // page], h, s % page]
                out["score"][b, h, d], out["pos"][b, h, d] = score[b, h, s], pos[b, h, s]
    return out


def check_evict(sg, cache, lens, seen, budget, recent):
    want = evicted(cache, lens, seen, budget, recent)
    new = sg.sage_kv_evict(cache, ints(lens), ints(seen), budget=budget, recent=recent)
    assert status(sg) == 0
    assert new.tolist() == [min(n, budget) for n in lens]
    for k, w in want.items():
        if w is not None:
            assert torch.equal(bits(getattr(cache, k).cpu()), bits(w)), k


EVICTS = [
    # H, d, page, budget, recent, lens
    (2, 64, 16, 40, 8, [100, 40, 41, 39, 0, 1]),
    (1, 128, 64, 1, 0, [2, 1, 300]),
    (3, 128, 32, 100, 100, [130, 101]),
    (1, 64, 16, 1000, 30, [1024, 1063, 1500]),
    (2, 64, 48, 2000, 100, [2100, 5000]),
]


@pytest.mark.parametrize("kind", ["fp16", "bf16", "int8", "fp8"])
@pytest.mark.parametrize("H,d,page,budget,recent,lens", EVICTS)
def test_evict(kind, H, d, page, budget, recent, lens):
    import bit_trainable_attention_sage_gb300 as sg
    B = len(lens)
    cache, _, _ = filled(kind, B, H, d, page, lens, seed=budget, score=True)
    g = torch.Generator().manual_seed(0)
    for b, n in enumerate(lens):
        for h in range(H):
            cache.pos[b, h, :n] = torch.randperm(max(n, 1) + 20, generator=g)[:n].int().cuda()
    check_evict(sg, cache, lens, [n + 20 for n in lens], budget, recent)


@pytest.mark.parametrize("case", ["ties", "all_equal", "special", "negative", "all_recent", "zeros"])
def test_evict_ties_and_special_scores(case):
    """Ties go to the lower slot; NaN last; -0 = +0; infinities and negative values in order."""
    import bit_trainable_attention_sage_gb300 as sg
    lens = [500, 137]
    cache, _, _ = filled("int8", 2, 2, 64, 16, lens, seed=3, score=True)
    g = torch.Generator().manual_seed(0)
    shape = cache.score.shape
    values = {"ties": torch.tensor([0.5, 0.25, 1.0]), "all_equal": torch.tensor([2.0]), "zeros": torch.tensor([0.0, -0.0]),
              "special": torch.tensor([float("nan"), float("inf"), float("-inf"), 0.0, -0.0, 1e-45, 1.0, -float("nan")]),
              "negative": torch.randn(300, generator=g), "all_recent": torch.rand(10, generator=g)}[case]
    cache.score.copy_(values[torch.randint(0, len(values), shape, generator=g)])
    cache.pos.copy_(torch.arange(shape[2], dtype=torch.int32).expand(shape))
    seen = [5, 2] if case == "all_recent" else lens
    check_evict(sg, cache, lens, seen, 100, 0 if case != "all_recent" else 50)


def test_evict_bad_pages_and_graph():
    """A move from or to a page that is none is left out and reported; a captured call replays."""
    import bit_trainable_attention_sage_gb300 as sg
    cache, _, _ = filled("bf16", 1, 1, 64, 16, [64], score=True, garbage=False)
    cache.score[0, 0, :64] = torch.arange(64, device="cuda").float()
    cache.table[0, 3] = 99999                             # the page of the best slots, 48 .. 63
    K = cache.K.clone()
    new = sg.sage_kv_evict(cache, ints([64]), ints([10 ** 6]), budget=16)
    assert status(sg) == 7 and new.tolist() == [16]
    assert torch.equal(cache.K, K)
    cache, _, _ = filled("bf16", 2, 2, 64, 16, [200, 150], score=True)
    lens, seen, first = ints([1, 1]), ints([10 ** 6, 10 ** 6]), [getattr(cache, k).clone() for k in ("K", "V", "score", "pos")]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        new = sg.sage_kv_evict(cache, lens, seen, budget=64)
    lens.copy_(ints([200, 150]))
    want = evicted(cache, [200, 150], [10 ** 6] * 2, 64, 0)
    graph.replay()
    assert new.tolist() == [64, 64]
    for k in ("K", "V", "score", "pos"):
        assert torch.equal(bits(getattr(cache, k).cpu()), bits(want[k]))
    assert not torch.equal(cache.K.view(torch.int16), first[0].view(torch.int16))


# ---- together -------------------------------------------------------------------------------


@pytest.mark.parametrize("kind", ["fp16", "int8", "fp8"])
def test_serving_loop(kind):
    """Prompt -> append (with the prompt's K mean in 8 bits) -> steps of turn, append, decode with
    weights, evict when over budget: every step against 64 bits over a plain list of rows."""
    import bit_trainable_attention_sage_gb300 as sg
    B, H, G, d, T, budget, recent = 2, 2, 3, 64, 64, 70, 10
    g = torch.Generator().manual_seed(0)
    rope = sg.make_rope(d, (16, 8, 8))
    cache = sg.make_kv_cache(B, H, d, 160, dtype=KINDS[kind], page=16, score=True)
    prompt = [torch.randn(B, H, T, d, generator=g).half().cuda() for _ in range(3)]
    positions = torch.arange(T, dtype=torch.int32, device="cuda").expand(3, 1, T).contiguous()
    _, Kp = sg.sage_rope(prompt[0], prompt[1], positions, rope)
    mu = sg.sage_quantize_smooth(prompt[0], Kp, prompt[2]).muK if kind != "fp16" else None
    lens = ints([T, T - 9])
    sg.sage_kv_append(cache, Kp, prompt[2], ints([0, 0]), count=lens, mu=mu)
    n = [T, T - 9]
    pos = [[list(range(n[b])) for _ in range(H)] for b in range(B)]
    score = [[[0.0] * n[b] for _ in range(H)] for b in range(B)]
    seen = list(n)

    def rows(b, h, pool, scale):
        at = torch.arange(n[b], device="cuda")
        p = cache.table[b, at // 16].long()
        x = pool.view(torch.int8)[p, h, at % 16].view(pool.dtype) if pool.element_size() == 1 else pool[p, h, at % 16]
        x = x.double()
        return (x if scale is None else x * scale[p, h, at % 16].double().unsqueeze(-1)).cpu().numpy()

    for step in range(30):
        q = torch.randn(B, H * G, 1, d, generator=g).half().cuda()
        k, v = (torch.randn(B, H, 1, d, generator=g).half().cuda() for _ in range(2))
        where = ints(seen)
        q, k = sg.sage_rope(q, k, where.view(1, B, 1).expand(3, B, 1).contiguous(), rope)
        sg.sage_kv_append(cache, k, v, lens, mu=mu, pos=where)
        lens = lens + 1
        n = [x + 1 for x in n]
        for b in range(B):
            for h in range(H):
                pos[b][h].append(seen[b])
                score[b][h].append(0.0)
        seen = [x + 1 for x in seen]
        was = cache.score.clone()
        O, L = sg.sage_attn_decode(q, cache, lens, score=True)
        Kr = [np.stack([rows(b, h, cache.K, cache.sK) for h in range(H)]) for b in range(B)]
        Vr = [np.stack([rows(b, h, cache.V, cache.sV) for h in range(H)]) for b in range(B)]
        check_decode(q, O, L, n, Kr, Vr, H, cache.score, was)
        # the last row is this step's token, in the cache's form
        if kind == "fp16":
            assert np.array_equal(Kr[0][:, -1], k[0, :, 0].double().cpu().numpy())
        for b in range(B):
            for h in range(H):
                score[b][h] = cache.score[b, h, :n[b]].tolist()
        if step % 8 == 7:
            for b in range(B):
                for h in range(H):
                    dst, src = evict64(score[b][h], pos[b][h], n[b], seen[b], budget, recent)
                    for i, j in zip(dst, src):
                        pos[b][h][i], score[b][h][i] = pos[b][h][j], score[b][h][j]
                    pos[b][h], score[b][h] = pos[b][h][:budget], score[b][h][:budget]
            lens = sg.sage_kv_evict(cache, lens, ints(seen), budget=budget, recent=recent)
            n = [min(x, budget) for x in n]
            assert lens.tolist() == n
            for b in range(B):
                for h in range(H):
                    assert cache.pos[b, h, :n[b]].tolist() == pos[b][h]
                    assert cache.score[b, h, :n[b]].tolist() == score[b][h]
    assert status(sg) == 0


def test_evict_long_rows_over_a_cluster():
    """Rows that a cluster shares, with ties across its parts, and rows too long for shared memory."""
    import bit_trainable_attention_sage_gb300 as sg
    for n, page, budget, levels in ((20000, 64, 7000, 0), (70000, 16, 60000, 40), (400000, 256, 1000, 0)):
        cap = -(-n // page) * page
        g = torch.Generator().manual_seed(n)
        pages = cap // page
        K = torch.randn(pages, 1, page, 64, generator=g).half().cuda()
        V = torch.randn(pages, 1, page, 64, generator=g).half().cuda()
        score = torch.rand(1, 1, cap, generator=g)
        if levels:
            score = (score * levels).floor()
        pos = torch.randperm(cap, generator=g).int().view(1, 1, cap)
        table = torch.randperm(pages, generator=g).int().view(1, pages)
        cache = sg.KvCache(K.clone(), V.clone(), table.cuda(), score=score.cuda(), pos=pos.cuda())
        recent = budget // 10
        new = sg.sage_kv_evict(cache, ints([n]), ints([cap]), budget=budget, recent=recent)
        assert status(sg) == 0 and new.tolist() == [budget]
        key = torch.where(pos[0, 0, :n] >= cap - recent, torch.tensor(float("inf")), score[0, 0, :n])
        stay = (-key).sort(stable=True).indices[:budget].sort().values
        src = stay[stay >= budget]
        gone = torch.ones(budget, dtype=torch.bool)
        gone[stay[stay < budget]] = False
        dst = gone.nonzero().flatten()
        score[0, 0, dst], pos[0, 0, dst] = score[0, 0, src], pos[0, 0, src]
        assert torch.equal(cache.score.cpu(), score) and torch.equal(cache.pos.cpu(), pos)
        t = table[0].long()
        for x, was in ((cache.K, K), (cache.V, V)):
            want = was.clone()
            want[t[dst // page].cuda(), 0, (dst % page).cuda()] = was[t[src // page].cuda(), 0, (src % page).cuda()]
            assert torch.equal(x, want)


@pytest.mark.parametrize("kind,Hq,H,d,page,lens", [
    ("int8", 4, 1, 64, 16, [9000, 130, 0, 2000]),         # every path of a long cache: shared, whole and empty pairs
    ("fp16", 40, 2, 128, 64, [5000, 1]),                  # three groups of heads a kv head
    ("bf16", 70, 1, 64, 128, [12000]),                    # more heads than are held at a time
    ("fp8", 6, 3, 128, 32, [64 * i for i in range(60, 0, -1)] + [7000]),
])
@pytest.mark.parametrize("score", [False, True])
def test_decode_long_caches(kind, Hq, H, d, page, lens, score):
    """Caches whose capacity takes the split path, with scores and without."""
    import bit_trainable_attention_sage_gb300 as sg
    q_dtype = KINDS[kind] if kind in ("fp16", "bf16") else torch.bfloat16
    cache, K, V = filled(kind, len(lens), H, d, page, lens, seed=Hq, score=score)
    Q = torch.randn(len(lens), Hq, 1, d, generator=torch.Generator().manual_seed(1)).to(q_dtype).cuda()
    was = cache.score.clone() if score else None
    O, L = sg.sage_attn_decode(Q, cache, ints(lens), score=score)
    assert status(sg) == 0
    check_decode(Q, O, L, lens, K, V, H, cache.score, was)


@pytest.mark.parametrize("B,page,n", [(5, 16, 0), (2000, 16, 3), (40, 64, 9000)])
def test_decode_mostly_empty_batches(B, page, n):
    """Rows without a token, a few with: a padded batch; O = 0 and L = -inf in all the others."""
    import bit_trainable_attention_sage_gb300 as sg
    lens = [0] * B
    if n:
        lens[B // 2], lens[B - 1] = n, 1
    cache, K, V = filled("fp16", B, 1, 64, page, lens, seed=B)
    Q = torch.randn(B, 3, 1, 64, generator=torch.Generator().manual_seed(1)).half().cuda()
    O, L = torch.full_like(Q, 7.0), torch.full((B, 3, 1), 7.0, device="cuda")
    sg.sage_attn_decode(Q, cache, ints(lens), out=O, lse=L)
    assert status(sg) == 0
    check_decode(Q, O, L, lens, K, V, 1)
