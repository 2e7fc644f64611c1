"""sage_attn_decode where the softmax is far from flat: a key that takes nearly all the weight and whose value
is small, values that are large and unattended.  What remains of the others has to keep its bits: the error of
an output is bounded relative to the sum of p |v|, however small p is (the bounds of cache_common, whose only
term for the probabilities themselves is 2^-17 of each)."""
import pytest
import torch

from tests.cache_common import KINDS, check_decode, codes_of

pytestmark = pytest.mark.gpu


def one_sequence(kind, K, V, page=64, seed=0):
    """A cache of one sequence and one kv head that holds the float32 rows K, V (n,d), and the rows as it holds
    them, in float64."""
    import bit_trainable_attention_sage_gb300 as sg
    n, d = K.shape
    m = -(-n // page)
    order = torch.randperm(m, generator=torch.Generator().manual_seed(seed))
    t = torch.arange(n)
    pools, scales, rows = [], [], []
    for x in (K, V):
        c, s = codes_of(x, kind) if kind in ("int8", "fp8") else (x.to(KINDS[kind]), None)
        pool = torch.zeros((m, 1, page, d), dtype=c.dtype)
        raw = (lambda y: y.view(torch.int8) if y.element_size() == 1 else y)  # noqa: E731
        raw(pool)[order[t // page], 0, t % page] = raw(c)
        scale = None
        if s is not None:
            scale = torch.zeros((m, 1, page))
            scale[order[t // page], 0, t % page] = s
        pools.append(pool.cuda())
        scales.append(None if scale is None else scale.cuda())
        rows.append((c.double() if s is None else c.double() * s.double().unsqueeze(-1)).numpy()[None])
    cache = sg.KvCache(pools[0], pools[1], order.int().view(1, m).cuda(), sK=scales[0], sV=scales[1],
                       score=torch.zeros((1, 1, m * page), device="cuda"))
    return cache, [rows[0]], [rows[1]]


def rows_of(n, d, heads, seed):
    """q (heads,d) near one direction, ordinary K and V (values near 1, of one sign, so that what is lost shows),
    and the direction: a key of `x` times it has a logit of about x sqrt(d)."""
    g = torch.Generator().manual_seed(seed)
    base = torch.where(torch.rand(d, generator=g) < 0.5, -1.0, 1.0)
    q = base + 0.1 * torch.randn(heads, d, generator=g)
    return q, torch.randn(n, d, generator=g), 1 + 0.3 * torch.randn(n, d, generator=g), base


def run(kind, q, K, V, score=False):
    import bit_trainable_attention_sage_gb300 as sg
    n, d = K.shape
    cache, Kr, Vr = one_sequence(kind, K, V)
    Q = q.to(KINDS[kind] if kind in ("fp16", "bf16") else torch.bfloat16).view(1, -1, 1, d).cuda()
    was = cache.score.clone() if score else None
    O, L = sg.sage_attn_decode(Q, cache, torch.tensor([n], dtype=torch.int32, device="cuda"), score=score)
    assert sg.sage_device_status() == 0
    check_decode(Q, O, L, [n], Kr, Vr, 1, cache.score if score else None, was)


@pytest.mark.parametrize("kind", ["fp16", "bf16", "int8", "fp8"])
@pytest.mark.parametrize("d,heads", [(64, 3), (128, 12)])
@pytest.mark.parametrize("n", [20, 1500, 20000])
@pytest.mark.parametrize("nats", [14, 18, 24, 30])
def test_sink_without_a_value(kind, d, heads, n, nats):
    """One key `nats` above the rest, its value zero: the output is what the others' small weights make of
    theirs.  (Values of 30000: fp16 outputs show them down to 30 nats.)"""
    q, K, V, base = rows_of(n, d, heads, nats)
    V *= 3e4 if kind == "fp16" else 1.0
    V.clamp_(-6e4, 6e4)
    at = n // 3
    K[at], V[at] = base * (nats / d ** 0.5), 0.0
    run(kind, q, K, V, score=n == 1500)


@pytest.mark.parametrize("kind", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("n", [60, 20000])
def test_sink_far_above(kind, n):
    """60 nats: weights of 2^-86, within float32 and so kept."""
    q, K, V, base = rows_of(n, 64, 2, 7)
    K[5], V[5] = base * (60 / 8), 0.0
    run(kind, q, K, V)


@pytest.mark.parametrize("kind", ["int8", "fp8", "bf16"])
@pytest.mark.parametrize("d,heads", [(64, 3), (128, 12)])
@pytest.mark.parametrize("n", [40, 1500, 20000])
@pytest.mark.parametrize("larger", [10, 16, 30])
@pytest.mark.parametrize("late", [False, True])
def test_large_values_without_weight(kind, d, heads, n, larger, late):
    """One value 2^larger times the others, its key 45 nats below the rest: it must not cost them their bits."""
    q, K, V, base = rows_of(n, d, heads, larger)
    at = n - 5 if late else 3
    K[at] = base * (-45 / d ** 0.5)
    V[at] *= 2.0 ** larger
    run(kind, q, K, V)


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("sink,larger", [(12, 7), (14, 5), (20, 12)])
@pytest.mark.parametrize("n", [200, 8192])
def test_sink_beside_large_values(kind, sink, larger, n):
    """Both at once: a sink without a value and a large value without weight."""
    q, K, V, base = rows_of(n, 128, 4, sink)
    K[0], V[0] = base * (sink / 128 ** 0.5), 0.0
    K[n // 2] = base * (-40 / 128 ** 0.5)
    V[n // 2] *= 2.0 ** larger
    run(kind, q, K, V)


@pytest.mark.parametrize("kind", ["int8", "fp8"])
def test_values_in_one_channel(kind):
    """A sink whose value stands in one channel only: in the others its codes are zero, and the small weights of
    the tokens beside it make the whole output."""
    q, K, V, base = rows_of(24, 64, 4, 1)
    K[0], V[0] = base * (20 / 8), 0.0
    V[0, 9] = 1e5
    run(kind, q, K, V)
