"""Several new tokens over 8-bit caches whose V scales are out of the ordinary: far below what a float's reciprocal holds,
far apart, and not finite.  The bounds are check_extend's."""
import numpy as np
import pytest
import torch

from tests.test_gpu_extend import cache_of, check_extend, ints
from tests.test_gpu_extend_edges import FEW, MANY, ONE, appended, both

pytestmark = pytest.mark.gpu

SHAPES = pytest.mark.parametrize("T,Hq", [FEW, ONE, MANY])
KINDS = pytest.mark.parametrize("kind,block", [("int8", 0), ("fp8", 0), ("int8", 16), ("fp8", 64)])
TYPES = pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])


def _sg():
    import bit_trainable_attention_sage_gb300 as sg
    return sg


def answers(kind, block, dtype, T, Hq, K, V, Q, d=64):
    """extend over a cache of K, V (1,2,n0 + T,d), appended in bf16, against 64 bits."""
    sg = _sg()
    n0 = K.shape[2] - T
    cache, Kd, Vd = appended(kind, d, 64, block, K.bfloat16().cuda(), V.bfloat16().cuda())
    O, L = sg.sage_attn_extend(Q, cache, ints([n0]))
    assert sg.sage_device_status() == 0
    if both(T, Hq) and dtype == torch.bfloat16 and max(float(np.abs(x).max()) for x in Vd) < 2.0 ** -110:
        check_below(O, L, Q, Kd[0], Vd[0], n0)
    else:
        check_extend(Q, O, L, [n0], [T], Kd, Vd, 2, both(T, Hq))
    return cache, O, L


def check_below(O, L, Q, K, V, n0):
    """Few rows, values below 2^-110 all of them: the two bf16 terms of p sV have 16 bits no longer.  bf16's smallest
    step is 2^-133, so each slot's p sV (its p at most 1) is off by at most 2^-134, times a code of at most 448; O is
    their sum over l.  The output's own half step is 2^-134 there or 2^-9 of it; a weight's other roundings are below 2^-12."""
    q, o, T, n = Q.double().cpu().numpy(), O.double().cpu().numpy(), Q.shape[2], K.shape[1]
    for h in range(Q.shape[1]):
        k, v = K[h * 2 // Q.shape[1]], V[h * 2 // Q.shape[1]]
        s = q[0, h] @ k.T / Q.shape[3] ** 0.5
        s[np.arange(n)[None, :] > n0 + np.arange(T)[:, None]] = -np.inf
        m = s.max(-1, keepdims=True)
        e = np.exp(s - m)
        l = e.sum(-1, keepdims=True)
        bound = n * 448 * 2.0 ** -134 / l + (2.0 ** -9 + 2.0 ** -11) * (e @ np.abs(v)) / l + 2.0 ** -134
        assert np.all(np.abs(o[0, h] - e @ v / l) <= bound)
        assert np.all(np.abs(L[0, h].double().cpu().numpy() - (m + np.log(l))[:, 0]) <= 2.0 ** -12)


@KINDS
@TYPES
@SHAPES
@pytest.mark.parametrize("where", ["one row", "a block", "half", "all"])
@pytest.mark.parametrize("size", [-131, -90, -61])
def test_small_scales(kind, block, dtype, T, Hq, where, size):
    """Values that leave a scale below 2^-128, whose reciprocal no float holds, or just above, beside ordinary ones or
    alone."""
    g = torch.Generator().manual_seed(7 + T)
    n, d = 500 + T, 64
    K, V = (torch.randn(1, 2, n, d, generator=g) for _ in range(2))
    V[:, :, {"one row": slice(131, 132), "a block": slice(128, 192), "half": slice(0, n // 2), "all": slice(None)}[where]] *= 2.0 ** size
    answers(kind, block, dtype, T, Hq, K, V, torch.randn(1, Hq, T, d, generator=g).to(dtype).cuda())


@KINDS
@SHAPES
@pytest.mark.parametrize("lead", [0.0, 8.0, 40.0])
def test_scales_far_apart(kind, block, T, Hq, lead):
    """Values from 2^-60 to 2^60, the small ones' logits ahead of the others'."""
    g = torch.Generator().manual_seed(8 + T)
    n, d = 600 + T, 64
    K, V = (torch.randn(1, 2, n, d, generator=g) * 0.25 for _ in range(2))
    level = (torch.arange(n) // 64 % 5 - 2).double()
    V *= torch.exp2(30 * level).float().view(1, 1, n, 1)
    K[..., 0] = (-lead * level * d ** 0.5 / 4).float()
    Q = torch.randn(1, Hq, T, d, generator=g)
    Q[..., 0] = 4.0
    answers(kind, block, torch.bfloat16, T, Hq, K, V, Q.bfloat16().cuda())


@KINDS
@TYPES
@SHAPES
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_sums_do_not_see_the_scales_of_v(kind, block, dtype, T, Hq, value):
    """A V scale that is not finite: O of the rows that see it is not, L is what it was, on every path."""
    sg = _sg()
    B, H, d, page, n0 = 2, 2, 64, 64, 300
    start = [n0, 0]
    cache, _, _ = cache_of(kind, B, H, d, page, block, [n0 + T, T], seed=T, garbage=False)
    Q = torch.randn(B, Hq, T, d).to(dtype).cuda()
    good_O, good_L = sg.sage_attn_extend(Q, cache, ints(start))
    # a row that all of sequence 0 sees, and one in the middle of sequence 1's new tokens
    G, slots = Hq // H, [70, T // 2]
    first = [0, max(0, T // 2 // block * block if block else T // 2)]
    for b, s in enumerate(slots):
        cache.sV[int(cache.table[b, s // page]), 1, s % page // (block or 1)] = value
    O, L = sg.sage_attn_extend(Q, cache, ints(start))
    assert torch.equal(O[:, :G], good_O[:, :G]) and torch.equal(L[:, :G], good_L[:, :G])
    assert L.isfinite().all() and torch.allclose(L, good_L, rtol=1e-6, atol=1e-5)
    for b in range(B):
        assert not O[b, G:, slots[b] if b else 0:].isfinite().any()
        assert O[b, G:, :first[b]].isfinite().all()
    assert sg.sage_device_status() == 0
