"""Slots that take a row's weight and carry no value or little: what the others carry still reaches an output in fp16."""
import numpy as np
import pytest
import torch

from tests.cache_common import U
from tests.test_gpu_extend import ints
from tests.test_gpu_extend_edges import MANY, ONE, appended

pytestmark = pytest.mark.gpu

FEW = (4, 4)


def _sg():
    import bit_trainable_attention_sage_gb300 as sg
    return sg


def check_rows(Q, O, L, n0, K, V, few, lost=2.0 ** -12):
    """As check_extend, but what fp16's range takes from the probabilities may be no more than `lost` of a row's largest
    output.  (One sequence.)"""
    _, Hq, T, d = Q.shape
    G, n = Hq // len(K), n0 + T
    eps = torch.finfo(Q.dtype).eps / 2
    tiny = 2.0 ** -25 if Q.dtype == torch.float16 else 2.0 ** -134
    o, lg, q = O[0].double().cpu().numpy(), L[0].double().cpu().numpy(), Q[0].double().cpu().numpy()
    hidden = np.arange(n)[None, :] > n0 + np.arange(T)[:, None]
    for h in range(Hq):
        k, v = K[h // G], V[h // G]
        s = q[h] @ k.T / np.sqrt(d)
        A = float((np.abs(q[h]) @ np.abs(k).T).max() / np.sqrt(d))
        s[hidden] = -np.inf
        m = s.max(-1, keepdims=True)
        e = np.exp(s - m)
        l = e.sum(-1, keepdims=True)
        p = e / l
        want, pv = p @ v, p @ np.abs(v)
        logit = (34 * (d // 16) + 8) * U * A + 4 * U * (2 * A * 1.4427 + 16)
        sums = (n / 16 + 400) * U
        rel = 2 * (logit + 2.0 ** -22) + 2 * sums + (n / 16 + 8) * 35 * U + (2.0 ** -17 if few else eps)
        bound = rel * pv + eps * np.abs(want) * (1 + rel) + tiny + (0.0 if few else lost * np.abs(want).max(-1, keepdims=True))
        err = np.abs(o[h] - want)
        assert np.all(err <= bound), (h, float((err / bound).max()), int((err / bound).max(-1).argmax()))
        assert np.all(np.abs(lg[h] - (m + np.log(l))[:, 0]) <= logit + sums + 2.0 ** -21 + 4 * U * (1 + np.abs(lg[h]).max()))


def made(n, d, sinks, lead, seed, size, dtype=torch.bfloat16):
    """K and V (1,2,n,d) with logits near 0 (q has 4 in channel 0), those of `sinks` ahead by `lead` nats; values of one
    sign near `size`."""
    g = torch.Generator().manual_seed(seed)
    K = torch.randn((1, 2, n, d), generator=g) * 0.02
    K[..., 0] = 0
    K[:, :, sinks, 0] = lead * d ** 0.5 / 4
    V = (1 + 0.25 * torch.randn((1, 2, n, d), generator=g).clamp(-3, 3)) * size
    return K.to(dtype).cuda(), V.to(dtype).cuda()


def queries(Hq, T, d, dtype, seed):
    Q = torch.randn((1, Hq, T, d), generator=torch.Generator().manual_seed(seed)) * 0.5
    Q[..., 0] = 4.0
    return Q.to(dtype).cuda()


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("block", [0, 16, 64])
@pytest.mark.parametrize("T,Hq", [FEW, ONE, MANY])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("lead", [6.0, 12.0, 18.0])
@pytest.mark.parametrize("at", [0, 2048])
def test_values_of_zero(kind, block, T, Hq, dtype, lead, at):
    """One block of slots, or one row, of no value and with nearly all the weight, over 4000 others."""
    sg = _sg()
    n0, d = 4000, 64
    sinks = slice(at, at + max(1, block))
    K, V = made(n0 + T, d, sinks, lead, 1, 0.25)
    V[:, :, sinks] = 0
    Q = queries(Hq, T, d, dtype, 2)
    cache, Kd, Vd = appended(kind, d, 64, block, K, V)
    O, L = sg.sage_attn_extend(Q, cache, ints([n0]))
    assert sg.sage_device_status() == 0
    check_rows(Q, O, L, n0, Kd[0], Vd[0], Hq // 2 * T <= 32)


def run(kind, dtype, block, T, Hq, n0, sinks, lead, size, *, d=64, change=None, seed=3):
    sg = _sg()
    K, V = made(n0 + T, d, sinks, lead, seed, size, dtype)
    V[:, :, sinks] = 0
    Q = queries(Hq, T, d, dtype, seed + 1)
    if change:
        change(K, V, Q)
    cache, Kd, Vd = appended(kind, d, 64, block, K, V)
    O, L = sg.sage_attn_extend(Q, cache, ints([n0]))
    assert sg.sage_device_status() == 0
    check_rows(Q, O, L, n0, Kd[0], Vd[0], Hq // 2 * T <= 32)
    return O


# a 16-bit pool, a scale a row, scales of blocks in which the sink is one row of many
POOLS = [("fp16", 0), ("int8", 0), ("int8", 16), ("fp8", 64)]


@pytest.mark.parametrize("kind,block", POOLS)
@pytest.mark.parametrize("T,Hq", [FEW, ONE, MANY])
@pytest.mark.parametrize("lead", [12.0, 18.0, 25.65, 33.0])
@pytest.mark.parametrize("n0", [200, 4096])
def test_one_slot_takes_the_weight(kind, block, T, Hq, lead, n0):
    """All others together carry an ordinary fp16 number, each far below 2^-25 of the largest probability."""
    O = run(kind, torch.float16, block, T, Hq, n0, slice(7, 8), lead, 6e4 / 1.75)
    if lead < 26 and n0 == 4096:
        assert bool((O > 1e-4).all())


@pytest.mark.parametrize("kind,block", POOLS)
@pytest.mark.parametrize("T,Hq", [ONE, MANY])
@pytest.mark.parametrize("carries", [1.0, 2.0 ** -6, 2.0 ** -14])
def test_the_slot_carries_little(kind, block, T, Hq, carries):
    """The slot with the weight has small values, or one value alone."""
    def small(K, V, Q):
        V[:, 0, 7] = carries
        V[:, 1, 7, 5] = carries
    run(kind, torch.float16, block, T, Hq, 3000, slice(7, 8), 25.65, 3e4, change=small)


@pytest.mark.parametrize("kind,block", POOLS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,Hq,n0", [(40, 2, 20000), (700, 6, 1000), (129, 2, 0), (256, 4, 256)])
def test_rows_that_need_it_among_rows_that_do_not(kind, block, d, T, Hq, n0):
    """Ranges of slots, tiles of several heads, and rows whose slot with the weight is another, or none."""
    def some(K, V, Q):
        Q[:, :, 1::3, 0] = 0.0
        Q[:, :, 2::3, 0] = -4.0
        K[:, :, n0 + 5::17, 0] = -25.0 * d ** 0.5 / 4
    run(kind, torch.float16, block, T, Hq, n0, slice(3, 4), 25.65, 2e4, d=d, change=some)


@pytest.mark.parametrize("T,Hq", [ONE, MANY])
def test_ragged_and_replayed(T, Hq):
    """Counts, a sequence without slots, and a graph whose replay needs the further walks where its capture did not."""
    sg = _sg()
    n0, d = 500, 64
    K, V = made(n0 + T, d, slice(9, 10), 25.65, 5, 3e4, torch.float16)
    V[:, :, 9] = 0
    cache = sg.make_kv_cache(3, 2, d, n0 + T, dtype=torch.float16, page=64)
    K3, V3 = (x.expand(3, -1, -1, -1).contiguous() for x in (K, V))
    sg.sage_kv_append(cache, K3, V3, ints([0] * 3))
    start, count = [n0, 0, 30], [T, 0, T - 3]
    Q = queries(Hq, T, d, torch.float16, 6).expand(3, -1, -1, -1).contiguous()
    easy = Q.clone()
    easy[..., 0] = 0
    held = easy.clone()
    s, c = ints(start), ints(count)
    sg.sage_attn_extend(held, cache, s, count=c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        O, L = sg.sage_attn_extend(held, cache, s, count=c)
    for x in (easy, Q, easy):
        held.copy_(x)
        graph.replay()
        again = sg.sage_attn_extend(x, cache, s, count=c)
        assert torch.equal(O, again[0]) and torch.equal(L, again[1])
        Kd, Vd = (y[0].double().cpu().numpy() for y in (K, V))
        for b in (0, 2):
            n = count[b]
            check_rows(x[b:b + 1, :, :n], O[b:b + 1, :, :n], L[b:b + 1, :, :n], start[b], Kd[:, :start[b] + n], Vd[:, :start[b] + n], False)
        assert bool((O[1] == 0).all()) and bool((O[2, :, T - 3:] == 0).all()) and bool(L[1].isneginf().all())
    assert sg.sage_device_status() == 0


@pytest.mark.parametrize("kind,block", POOLS)
@pytest.mark.parametrize("T,Hq", [ONE, MANY])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_values_that_are_not_finite_show(kind, block, T, Hq, value):
    """Beside a slot that takes the weight: rows that see such a value or scale show it, the others are as they would be
    without it, and L does not depend on it."""
    sg = _sg()
    n0, d, s = 700, 64, 700 + T // 2
    K, V = made(n0 + T, d, slice(7, 8), 25.65, 9, 3e4, torch.float16)
    V[:, :, 7] = 0
    Q = queries(Hq, T, d, torch.float16, 10)
    cache, Kd, Vd = appended(kind, d, 64, block, K, V)
    good_O, good_L = sg.sage_attn_extend(Q, cache, ints([n0]))
    check_rows(Q, good_O, good_L, n0, Kd[0], Vd[0], False)
    p, off, size = int(cache.table[0, s // 64]), s % 64, block or 1
    if cache.sV is None:
        cache.V[p, 1, off, 3] = value
    else:
        cache.sV[p, 1, off // size] = value
    O, L = sg.sage_attn_extend(Q, cache, ints([n0]))
    G, before = Hq // 2, max(0, s // size * size - n0)
    assert torch.equal(O[:, :G], good_O[:, :G]) and torch.allclose(L, good_L, rtol=1e-6, atol=1e-5)
    reached = O[:, G:, T // 2:] if cache.sV is not None else O[:, G:, T // 2:, 3]
    assert not reached.isfinite().any()
    assert torch.allclose(O[:, G:, :before].float(), good_O[:, G:, :before].float(), rtol=2.0 ** -9, atol=2.0 ** -20)
    assert sg.sage_device_status() == 0
