"""Calls of the position and cache operators that their documents allow or refuse, as a program makes them."""
import pytest
import torch

from tests.cache_common import check_decode, filled

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_decode_ignores_a_workspace_it_does_not_need():
    """A short cache without scores needs none: one that starts anywhere, or is too small, is no fault."""
    import bit_trainable_attention_sage_gb300 as sg
    lens = [100, 7]
    cache, K, V = filled("int8", 2, 1, 64, 16, lens, score=True)
    Q = torch.randn(2, 4, 1, 64, generator=torch.Generator().manual_seed(0)).half().cuda()
    assert sg.lib().sage_decode_workspace_bytes(cache._struct(Q, "Q"), 4, 0) == 0
    buf = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    for ws in (buf[16:], buf[48:64], buf[1:2]):
        O, L = sg.sage_attn_decode(Q, cache, ints(lens), workspace=ws)
        check_decode(Q, O, L, lens, K, V, 1)
    assert sg.sage_device_status() == 0
    with pytest.raises(sg.SageError):                     # scores need one, and it begins at a multiple of 256
        sg.sage_attn_decode(Q, cache, ints(lens), score=True, workspace=buf[16:])
    was = cache.score.clone()
    O, L = sg.sage_attn_decode(Q, cache, ints(lens), score=True, workspace=buf[256:])
    check_decode(Q, O, L, lens, K, V, 1, cache.score, was)
