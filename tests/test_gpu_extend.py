"""Attention of several new tokens a sequence over the cache, against 64 bits."""
import numpy as np
import pytest
import torch

from tests.block_common import filled_blocks
from tests.cache_common import U, filled

pytestmark = pytest.mark.gpu


def _sg():
    import bit_trainable_attention_sage_gb300 as sg
    return sg


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cache_of(kind, B, H, d, page, block, lens, **kw):
    if block:
        return filled_blocks(kind, B, H, d, page, block, lens, **kw)
    return filled(kind, B, H, d, page, lens, **kw)


def check_extend(Q, O, L, start, count, K, V, H, few):
    """Every output of a call against 64 bits.

    A logit is d / 16 tensor-core sums of 16 products and the running sum, each term cut at 2^-23 of the
    largest: 34 u of A = sum |q k| / sqrt(d) a step, and three roundings of scales; the exponent's difference
    and log2 of V's scale round by 4 u of their sizes (below 2 A log2 e + 16).  A weight moves by twice the largest logit error.
    Sums of exponentials: n / 16 + 400 roundings of positive terms.  The second product: n / 16 sums, 34 u each, a
    rescaling u each.  Probabilities: 2^-17 (few rows: two terms), else rounded to half a step of the type, and in fp16
    off by 2^-36 of the largest p sV (a code is below 2^9 scales, so of 2^9 the largest p |v| a slot)."""
    B, Hq, T, d = Q.shape
    G = Hq // H
    eps = torch.finfo(Q.dtype).eps / 2
    tiny = 2.0 ** -25 if Q.dtype == torch.float16 else 2.0 ** -134
    o, lg, q = O.double().cpu().numpy(), L.double().cpu().numpy(), Q.double().cpu().numpy()
    err2 = ref2 = 0.0
    for b in range(B):
        n, c = start[b] + count[b], count[b]
        assert np.all(o[b, :, c:] == 0) and np.all(lg[b, :, c:] == -np.inf), b
        if c == 0:
            continue
        hidden = np.arange(n)[None, :] > start[b] + np.arange(c)[:, None]
        for h in range(Hq):
            k, v = K[b][h // G], V[b][h // G]
            s = q[b, h, :c] @ k.T / np.sqrt(d)
            A = float((np.abs(q[b, h, :c]) @ np.abs(k).T).max() / np.sqrt(d))
            s[hidden] = -np.inf
            m = s.max(-1, keepdims=True)
            e = np.exp(s - m)
            l = e.sum(-1, keepdims=True)
            p = e / l
            want, Lw = p @ v, (m + np.log(l))[:, 0]
            pv = p @ np.abs(v)
            logit = (34 * (d // 16) + 8) * U * A + 4 * U * (2 * A * 1.4427 + 16)
            weight = 2 * (logit + 2.0 ** -22)
            sums = (n / 16 + 400) * U
            rel = weight + 2 * sums + (n / 16 + 8) * 35 * U + (2.0 ** -17 if few else eps)
            low = 0.0 if few or Q.dtype != torch.float16 else n * 2.0 ** -36 * 2.0 ** 9 * float((p * np.abs(v).max(-1)).max())
            err = np.abs(o[b, h, :c] - want)
            bound = rel * pv + eps * np.abs(want) * (1 + rel) + low + tiny
            assert np.all(err <= bound), (b, h, float((err / bound).max()), int((err / bound).max(-1).argmax()))
            assert np.all(np.abs(lg[b, h, :c] - Lw) <= logit + sums + 2.0 ** -21 + 4 * U * (1 + np.abs(Lw).max())), (b, h)
            err2 += float((err ** 2).sum())
            ref2 += float((want ** 2).sum())
    # random values: roundings of p and of O each add about 0.4 of a half step in the mean square
    assert err2 <= (2 * eps) ** 2 * ref2 + 1e-30, (err2 / max(ref2, 1e-300)) ** 0.5


def run(kind, dtype, d, page, block, start, count, H, Hq, T, **kw):
    sg = _sg()
    B = len(start)
    cache, K, V = cache_of(kind, B, H, d, page, block, [s + c for s, c in zip(start, count)], **kw)
    Q = torch.randn(B, Hq, T, d).to(dtype).cuda()
    for b, c in enumerate(count):
        Q[b, :, c:] = float("nan")
    O, L = sg.sage_attn_extend(Q, cache, ints(start), count=None if all(c == T for c in count) else ints(count))
    assert sg.sage_device_status() == 0
    check_extend(Q, O, L, start, count, K, V, H, Hq // H * T <= 32)
    return Q, O, L


FORMS = [("int8", torch.bfloat16, 128, 64, 64), ("fp8", torch.float16, 64, 48, 16), ("int8", torch.float16, 128, 16, 0),
         ("fp8", torch.bfloat16, 64, 64, 0), ("fp16", torch.float16, 128, 64, 0), ("bf16", torch.bfloat16, 64, 16, 0),
         ("int8", torch.bfloat16, 64, 128, 32), ("fp8", torch.bfloat16, 128, 32, 32)]


@pytest.mark.parametrize("kind,dtype,d,page,block", FORMS)
@pytest.mark.parametrize("T,Hq", [(1, 2), (3, 4), (4, 16), (7, 6)])
def test_few_rows(kind, dtype, d, page, block, T, Hq):
    run(kind, dtype, d, page, block, [0, 1, 15, 130, 517, 64, 2000], [T, T, 0, T, max(1, T - 1), 1, T], 2, Hq, T, seed=T)


@pytest.mark.parametrize("kind,dtype,d,page,block", FORMS)
@pytest.mark.parametrize("T,Hq,start,count", [
    (33, 2, [0, 1, 95, 300], [33, 32, 33, 0]), (64, 6, [64, 0, 1000], [64, 1, 63]), (128, 2, [0, 128], [128, 128]), (130, 4, [126, 700], [130, 7]),
    (300, 2, [0, 511], [300, 299])])
def test_many_rows(kind, dtype, d, page, block, T, Hq, start, count):
    run(kind, dtype, d, page, block, start, count, 2, Hq, T, seed=T)


@pytest.mark.parametrize("kind,dtype,d,page,block", FORMS)
def test_split_slots(kind, dtype, d, page, block):
    """Few tiles over long caches: ranges of slots, some of them empty."""
    run(kind, dtype, d, page, block, [9000, 3, 0], [40, 40, 0], 1, 2, 40, seed=3)


@pytest.mark.parametrize("kind,dtype,d,page,block", FORMS[:4])
def test_whole_tiles(kind, dtype, d, page, block):
    run(kind, dtype, d, page, block, [300], [512], 2, 6, 512, seed=4)
