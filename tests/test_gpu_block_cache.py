"""The cache with one scale for each block of rows: append against the definition bit for bit, one-token
attention over it against 64 bits."""
import pytest
import torch

from tests.block_common import STORE, append_blocks, filled_blocks
from tests.cache_common import check_decode

pytestmark = pytest.mark.gpu


def _sg():
    import bit_trainable_attention_sage_gb300 as sg
    return sg


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def bits(t):
    return t.contiguous().view(torch.int32) if t.dtype == torch.float32 else t.contiguous().view(torch.int8)


def state(cache):
    """The pools on the CPU: codes as float32 values, scales."""
    return [(c.cpu().float(), s.cpu()) for c, s in ((cache.K, cache.sK), (cache.V, cache.sV))]


def check_append(cache, kind, K, V, start, count, mu=None, **kw):
    """One call against the definition, the whole pool of it."""
    sg = _sg()
    want = state(cache)
    xs = [K.cpu().float(), V.cpu().float()]
    if mu is not None:
        xs[0] = xs[0] - mu.cpu().unsqueeze(2)
    for (c, s), x in zip(want, xs):
        append_blocks(c, s, cache.table.cpu(), x, start, count, cache.block, kind)
    sg.sage_kv_append(cache, K, V, ints(start), count=ints(count), mu=mu, **kw)
    assert sg.sage_device_status() == 0
    for (c, s), code, scale in zip(want, (cache.K, cache.V), (cache.sK, cache.sV)):
        assert torch.equal(bits(scale.cpu()), bits(s))
        assert torch.equal(code.cpu().float(), c)


@pytest.mark.parametrize("kind,dtype,d,page,block,smooth", [
    ("int8", torch.bfloat16, 128, 64, 64, True), ("int8", torch.float16, 64, 64, 32, False), ("fp8", torch.bfloat16, 64, 64, 64, True),
    ("fp8", torch.float16, 128, 48, 16, False), ("int8", torch.bfloat16, 64, 16, 16, True), ("fp8", torch.bfloat16, 128, 96, 32, True),
    ("int8", torch.float16, 128, 128, 64, False), ("fp8", torch.float16, 64, 128, 64, False)])
def test_append(kind, dtype, d, page, block, smooth):
    """Prompts, then chunks and single tokens that go on in the middle of blocks, ragged, some of none."""
    B, H = 5, 3
    cache, _, _ = filled_blocks(kind, B, H, d, page, block, [0] * B, room=400, garbage=False, seed=d + block)
    g = torch.Generator().manual_seed(7)
    new = lambda T, v: (torch.randn((B, H, T, d), generator=g) * v).to(dtype).cuda()  # noqa: E731
    mu = torch.randn((B, H, d), generator=g).cuda() * 2 if smooth else None
    start = [0] * B
    for T, count, v in ((150, [150, 1, 0, 64, 63], 1.0), (1, [1] * B, 0.3), (1, [1, 1, 0, 1, 1], 4.0), (33, [33, 32, 31, 1, 0], 1.5),
                        (1, [1] * B, 16.0), (2, [2, 2, 1, 0, 2], 1e-3), (90, [90, 65, 64, 63, 16], 30.0), (7, [7] * B, 64.0)):
        check_append(cache, kind, new(T, v), new(T, v), start, count, mu)
        start = [s + c for s, c in zip(start, count)]


@pytest.mark.parametrize("kind", ["int8", "fp8"])
def test_append_single_tokens_fill_a_block(kind):
    """64 steps of one token: the block's scale is that of all its rows, and each code within a step for every time it grew."""
    sg = _sg()
    H, d, block = 2, 64, 64
    cache, _, _ = filled_blocks(kind, 1, H, d, 64, block, [0], room=64, garbage=False)
    K = (torch.randn(1, H, block, d) * torch.linspace(0.5, 2, block).view(1, 1, block, 1)).bfloat16().cuda()
    for t in range(block):
        check_append(cache, kind, K[:, :, t:t + 1].contiguous(), -K[:, :, t:t + 1].contiguous(), [t], [1])
    page = int(cache.table[0, 0])
    top = K.float().abs().amax((-1, -2))[0] / torch.full((1,), 127.0 if kind == "int8" else 448.0, device="cuda")
    assert torch.equal(cache.sK[page, :, 0], top) and torch.equal(cache.sV[page, :, 0], top)
    got = cache.K[page].float() * cache.sK[page].unsqueeze(-1)
    step = cache.sK[page].unsqueeze(-1) / 2 if kind == "int8" else K[0].float().abs() * 2.0 ** -4 + cache.sK[page].unsqueeze(-1) * 2.0 ** -10
    # the scale grew at most 63 times; roundings add
    assert bool(((got - K[0].float()).abs() <= 64 * step * (1 + 2.0 ** -4) ** (0 if kind == "int8" else 64)).all())
    assert sg.sage_device_status() == 0


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("d", [64, 128])
def test_append_unusual_values(kind, d):
    """Zero blocks, a zero block that goes on with values, tiny and huge scales, -0."""
    H, block = 2, 16
    cache, _, _ = filled_blocks(kind, 1, H, d, 32, block, [0], room=128, garbage=False)
    z = torch.zeros(1, H, 20, d, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(1, H, 20, d).bfloat16().cuda()
    check_append(cache, kind, z, -z, [0], [20])
    check_append(cache, kind, x[:, :, :3].contiguous(), z[:, :, :3].contiguous(), [20], [3])       # from a scale of 0
    for i, v in enumerate((2.0 ** -120, 2.0 ** -130, 2.0 ** 100, 2.0 ** 120)):
        check_append(cache, kind, x * v, x * -v, [32], [20])
        check_append(cache, kind, x * v * 3, x * v * 5, [52], [20])


@pytest.mark.parametrize("kind", ["int8", "fp8"])
def test_append_not_finite(kind):
    """A NaN or an infinity shows in its block's scale, and in no other block's."""
    sg = _sg()
    cache, _, _ = filled_blocks(kind, 2, 2, 64, 32, 16, [0, 0], room=64, garbage=False)
    K, V = (torch.randn(2, 2, 48, 64).half().cuda() for _ in range(2))
    K[0, 1, 20, 5], V[1, 0, 47, 63] = float("nan"), float("-inf")
    sg.sage_kv_append(cache, K, V, ints([0, 0]))
    sK = cache.sK[cache.table[:, :2].long()].permute(0, 2, 1, 3).flatten(2)       # (B, H, blocks)
    sV = cache.sV[cache.table[:, :2].long()].permute(0, 2, 1, 3).flatten(2)
    bad_k, bad_v = torch.zeros(2, 2, 3, dtype=torch.bool), torch.zeros(2, 2, 3, dtype=torch.bool)
    bad_k[0, 1, 1] = bad_v[1, 0, 2] = True
    assert torch.equal(~sK.cpu()[..., :3].isfinite(), bad_k) and torch.equal(~sV.cpu()[..., :3].isfinite(), bad_v)
    # a row that follows does not hide it
    sg.sage_kv_append(cache, K[:, :, :1].contiguous(), V[:, :, :1].contiguous(), ints([31, 47]))
    assert cache.sK[int(cache.table[0, 0]), 1, 1].isnan() and cache.sV[int(cache.table[1, 1]), 0, 0].isinf()
    assert sg.sage_device_status() == 0


def test_append_out_of_range():
    """Slots and pages out of range are left out and reported; the rest is written."""
    sg = _sg()
    cache, _, _ = filled_blocks("int8", 3, 2, 64, 32, 16, [0, 0, 0], room=64, garbage=False)
    cap = cache.capacity
    K = torch.randn(3, 2, 40, 64).bfloat16().cuda()
    cache.table[1, 0] = cache.pages
    cache.table[2, 2] = int(cache.table[0, 1])                  # the third page of sequence 2: never a slot of this call
    was = cache.K.clone()
    sg.sage_kv_append(cache, K, K, ints([-20, 0, cap - 32 - 32]))
    assert sg.sage_device_status() == 7 and sg.sage_device_status() == 0
    # sequence 0: tokens 20.. at slots 0..; 1: page 0 is none, tokens 32.. in its second page; 2: all 40
    p0, p1 = int(cache.table[0, 0]), int(cache.table[1, 1])
    s = K[0, :, 20:36].float().abs().amax((-1, -2)) / torch.full((1,), 127.0, device="cuda")
    assert torch.equal(cache.sK[p0, :, 0], s)
    assert torch.equal(cache.sK[p1, :, 0], K[1, :, 32:].float().abs().amax((-1, -2)) / torch.full((1,), 127.0, device="cuda"))
    named = set(cache.table.flatten().tolist())
    for p in set(range(cache.pages)) - named:
        assert torch.equal(cache.K[p], was[p])
    sg.sage_kv_append(cache, K, K, ints([cap - 8, cap, 1 << 30]))
    assert sg.sage_device_status() == 7


def test_append_counts_out_of_range():
    sg = _sg()
    cache, _, _ = filled_blocks("fp8", 2, 1, 64, 16, 16, [0, 0], room=32, garbage=False)
    K = torch.randn(2, 1, 4, 64).half().cuda()
    was = cache.K.clone()
    sg.sage_kv_append(cache, K, K, ints([0, 0]), count=ints([-3, 9]))       # none, and all 4
    assert sg.sage_device_status() == 7
    assert torch.equal(bits(cache.K[int(cache.table[0, 0])]), bits(was[int(cache.table[0, 0])]))
    assert int((bits(cache.K) != bits(was)).any(-1).sum()) == 4


@pytest.mark.parametrize("kind,dtype,d,page,block", [
    ("int8", torch.bfloat16, 128, 64, 64), ("fp8", torch.float16, 64, 48, 16), ("int8", torch.float16, 64, 128, 32), ("fp8", torch.bfloat16, 128, 16, 16)])
@pytest.mark.parametrize("lens,Hq", [([0, 1, 15, 16, 17, 63, 64, 65, 129, 500], 3), ([2000, 3, 0, 700], 24), ([300] * 300, 6), ([9000], 48)])
def test_decode(kind, dtype, d, page, block, lens, Hq):
    sg = _sg()
    B, H = len(lens), 3
    cache, K, V = filled_blocks(kind, B, H, d, page, block, lens, seed=len(lens) + d)
    Q = torch.randn(B, Hq, 1, d).to(dtype).cuda()
    O, L = sg.sage_attn_decode(Q, cache, ints(lens))
    assert sg.sage_device_status() == 0
    check_decode(Q, O, L, lens, K, V, H)


def test_decode_long_and_shared():
    """One sequence past every split, and another that shares its first pages."""
    sg = _sg()
    lens = [40000, 20010]
    cache, K, V = filled_blocks("int8", 2, 2, 64, 64, 64, lens, seed=3, shared=[(1, 0, 300)])
    Q = torch.randn(2, 8, 1, 64).bfloat16().cuda()
    O, L = sg.sage_attn_decode(Q, cache, ints(lens))
    check_decode(Q, O, L, lens, K, V, 2)


def test_decode_scale_of_a_block_is_not_finite():
    """A block whose scale is NaN reaches the heads that read it, and no other."""
    sg = _sg()
    cache, K, V = filled_blocks("fp8", 2, 2, 64, 32, 32, [70, 70], seed=5)
    Q = torch.randn(2, 4, 1, 64).half().cuda()
    cache.sK[int(cache.table[0, 1]), 1, 0] = float("nan")
    cache.sV[int(cache.table[1, 2]), 0, 0] = float("inf")
    O, L = sg.sage_attn_decode(Q, cache, ints([70, 70]))
    assert O[0, 2:].isnan().all() and L[0, 2:].isnan().all() and not O[1, :2].isfinite().any()
    assert O[0, :2].isfinite().all() and O[1, 2:].isfinite().all() and L[1].isfinite().all()


def test_a_loop_of_append_and_decode_in_a_graph():
    """Steps of one token captured and replayed, against the same steps made one by one."""
    sg = _sg()
    B, H, d = 3, 2, 128
    caches = [filled_blocks("int8", B, H, d, 32, 32, [5, 31, 64], room=40, seed=9)[0] for _ in range(2)]
    K, V, Q = (torch.empty(B, H, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    Q = torch.empty(B, 4, 1, d, dtype=torch.bfloat16, device="cuda")
    lens = [ints([5, 31, 64]) for _ in range(2)]
    one = ints([1] * B)

    def step(i):
        sg.sage_kv_append(caches[i], K, V, lens[i])
        lens[i] += one
        return sg.sage_attn_decode(Q, caches[i], lens[i])
    for t in (K, V, Q):
        t.normal_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(0)
    lens[0].copy_(ints([5, 31, 64]))
    for n in range(36):
        for t in (K, V, Q):
            t.normal_()
        K *= 1 + n % 7
        graph.replay()
        O, L = step(1)
        assert torch.equal(O, out[0]) and torch.equal(L, out[1])
    assert all(torch.equal(bits(a), bits(b)) for a, b in ((caches[0].K, caches[1].K), (caches[0].V, caches[1].V)))
    assert all(STORE["int8"] == c.K.dtype for c in caches) and sg.sage_device_status() == 0
