"""Drafts that are taken back from a block with one scale: what stays of them is what the interface says."""
import pytest
import torch

from tests.block_common import TOP, append_blocks, quotients
from tests.test_gpu_extend import ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,dtype", [("int8", torch.int8), ("fp8", torch.float8_e4m3fn)])
@pytest.mark.parametrize("block", [16, 64])
def test_a_rejected_outlier_stays_in_the_scale(kind, dtype, block):
    """Rows, then a large draft in the same block, taken back and overwritten: codes and scales are those of the rule that a
    block's scale only grows."""
    import bit_trainable_attention_sage_gb300 as sg
    g = torch.Generator().manual_seed(block)
    H, d, page = 2, 64, 64
    cache = sg.make_kv_cache(1, H, d, 128, dtype=dtype, page=page, block=block)
    x = torch.randn(1, H, 10, d, generator=g).bfloat16()
    draft = 20 * torch.randn(1, H, 3, d, generator=g).bfloat16()
    new = torch.randn(1, H, 2, d, generator=g).bfloat16()
    pool, scale = torch.zeros(cache.pages, H, page, d), torch.zeros(cache.pages, H, page // block)
    table = cache.table.cpu()
    for rows, at in ((x, 0), (draft, 10), (new, 10)):
        sg.sage_kv_append(cache, rows.cuda(), rows.cuda(), ints([at]))
        append_blocks(pool, scale, table, rows.float(), [at], [rows.shape[2]], block, kind)
    p = int(table[0, 0])
    for k, s in ((cache.K, cache.sK), (cache.V, cache.sV)):
        assert torch.equal(s[p].cpu(), scale[p]) and torch.equal(k[p, :, :12].cpu().float(), pool[p, :, :12])
    assert bool((scale[p, :, 0] == draft[0].float().abs().amax((-1, -2)) / torch.full((1,), TOP[kind])).all())
    assert sg.sage_device_status() == 0
    # a call that begins the block takes its scale from its own rows
    sg.sage_kv_append(cache, x.cuda(), x.cuda(), ints([0]))
    s = x[0].float().abs().amax((-1, -2)) / torch.full((1,), TOP[kind])
    assert torch.equal(cache.sK[p, :, 0].cpu(), s)
    assert torch.equal(cache.K[p, :, :10].cpu().float(), quotients(x[0].float(), s.view(-1, 1, 1), kind))
