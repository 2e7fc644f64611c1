"""Values in K or V that are not finite: every row that sees one shows it."""
import numpy as np
import pytest
import torch

from tests.test_gpu_extend import cache_of, ints
from tests.test_gpu_extend_edges import FEW, FORMS, MANY, ONE

pytestmark = pytest.mark.gpu


def _sg():
    import bit_trainable_attention_sage_gb300 as sg
    return sg


def codes(pool, table, n, page):
    """A pool's rows (heads, n, d) of the sequence of this row of the table, as float64 without scales."""
    s = torch.arange(n, device=pool.device)
    x = pool.view(torch.int8)[table[s // page].long(), :, s % page].view(pool.dtype) if pool.element_size() == 1 else pool[table[s // page].long(), :, s % page]
    return x.double().permute(1, 0, 2)


@pytest.mark.parametrize("kind,dtype,d,page,block", FORMS)
@pytest.mark.parametrize("T,Hq", [FEW, ONE, MANY])
@pytest.mark.parametrize("slot", [3, 70, -1])
def test_every_row_that_sees_it(kind, dtype, d, page, block, T, Hq, slot):
    """A NaN or an infinity in a slot that all rows see, and in the middle of the new tokens.  In V or its scale, and a NaN in K
    or its scale, no row that sees it is finite.  An infinity in K or its scale makes a logit plus or minus infinity or NaN:
    minus infinity takes the slot out, the others leave no number."""
    sg = _sg()
    n0, G = 100, Hq // 2
    s = slot if slot >= 0 else n0 + T // 2
    cache, _, _ = cache_of(kind, 1, 2, d, page, block, [n0 + T], seed=T, garbage=False)
    Q = torch.randn(1, Hq, T, d).to(dtype).cuda()
    good_O, good_L = sg.sage_attn_extend(Q, cache, ints([n0]))
    p, off = int(cache.table[0, s // page]), s % page
    t = torch.arange(T, device="cuda")
    size = block if cache.sK is not None and block else 1
    s0 = s // size * size                                          # the slots that the value reaches
    for what in ("K", "V"):
        pool, scale = (cache.K, cache.sK) if what == "K" else (cache.V, cache.sV)
        for value in (float("nan"), float("inf")):
            at = pool[p, 1, off, 3:4] if scale is None else scale[p, 1, off // size:off // size + 1]
            was = at.clone()
            at.fill_(value)
            O, L = sg.sage_attn_extend(Q, cache, ints([n0]))
            assert torch.equal(O[:, :G], good_O[:, :G]) and torch.equal(L[:, :G], good_L[:, :G])
            O, L, q = O[0, G:], L[0, G:], Q[0, G:].double()
            if what == "V":
                sees = n0 + t >= s0
                reached = O[:, sees] if scale is not None else O[:, sees, 3]
                assert not reached.isfinite().any()
                assert L.isfinite().all()
            elif value != value:
                assert O[:, n0 + t >= s].isnan().all() and L[:, n0 + t >= s].isnan().all()
                assert O[:, n0 + t >= s0].isnan().all()
            else:
                rows = codes(cache.K, cache.table[0], n0 + T, page)[1, s0:s0 + size]
                x = q @ (rows if scale is not None else rows.nan_to_num(posinf=1e30)).T        # (G, T, size): the sign of the logit
                if scale is None:
                    x = torch.where(q[..., 3:4] == 0, torch.nan, x)
                seen = (n0 + t).view(-1, 1) >= s0 + torch.arange(rows.shape[0], device="cuda")
                lost = (seen & ~(x < 0)).any(-1)
                assert O[lost].isnan().all() and not L[lost].isfinite().any()
                assert O[~lost].isfinite().all() and L[~lost].isfinite().all()
                if scale is None or size == 1:
                    rest = ~lost & (n0 + t < s)                    # (and rows before it are as they were)
                    assert torch.allclose(O[rest].float(), good_O[0, G:][rest].float(), rtol=2.0 ** -6, atol=1e-3)
            at.copy_(was)
    assert sg.sage_device_status() == 0
