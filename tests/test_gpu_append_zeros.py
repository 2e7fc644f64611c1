"""Zeros of either sign in sage_kv_append: E4M3 has both, and the nearest code of fl32(x / delta) keeps the
sign; INT8 has one; rows of zeros alone are code 0."""
import pytest
import torch

from tests.cache_common import KINDS, codes_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("mu", [False, True])
def test_zeros_keep_their_sign(kind, dtype, d, mu):
    import bit_trainable_attention_sage_gb300 as sg
    T = 50
    g = torch.Generator().manual_seed(d)
    K, V = (torch.randn(1, 2, T, d, generator=g).to(dtype) for _ in range(2))
    for x in (K, V):
        hit = torch.rand(x.shape, generator=g) < 0.3
        x[hit] = torch.where(torch.rand(int(hit.sum()), generator=g) < 0.5, -0.0, 0.0).to(dtype)
        x[:, :, 7] = -0.0                                   # a row of zeros: scale 0, codes 0
    mu_t = torch.randn(1, 2, d, generator=g) if mu else None
    if mu:
        mu_t[:, :, ::2] = 0.0
        mu_t[:, :, ::4] = -0.0                              # x - mu is -0 only for -0 - +0
    cache = sg.make_kv_cache(1, 2, d, T, dtype=KINDS[kind])
    sg.sage_kv_append(cache, K.cuda(), V.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda"), mu=None if mu_t is None else mu_t.cuda())
    for x, pool, scale in ((K.float() - (mu_t.unsqueeze(2) if mu else 0.0), cache.K, cache.sK), (V.float(), cache.V, cache.sV)):
        codes, s = codes_of(x, kind)
        assert kind == "int8" or (codes.view(torch.int8) == -128).any()
        assert torch.equal(scale[0, :, :T].cpu(), s[0])
        assert torch.equal(pool.view(torch.int8)[0, :, :T].cpu(), codes.view(torch.int8)[0])
