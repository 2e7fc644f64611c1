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
