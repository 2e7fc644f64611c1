"""Sequences that together want more pages than 32 bits count."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_more_wanted_than_32_bits_count():
    """32800 sequences of 65600 pages each over a pool of 1000: the first gets what there is, and the rest, whose places lie
    past 2^31, nothing."""
    import bit_trainable_attention_sage_gb300 as sg
    B, M, page, pages = 32800, 65600, 16, 1000
    assert B * M > 1 << 31
    ints = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    K, V = (torch.zeros(pages, 1, page, 64, dtype=torch.half, device="cuda") for _ in range(2))
    table = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
    cache = sg.KvCache(K, V, table, refs=ints(pages), held=ints(B))
    # the first sequences hold pages already
    few = ints(B)
    few[:5] = 3 * page
    assert sg.sage_kv_resize(cache, few)[:6].tolist() == [3 * page] * 5 + [0]
    want = torch.full((B,), M * page, dtype=torch.int32, device="cuda")
    slots = sg.sage_kv_resize(cache, want)
    assert [sg.sage_device_status() for _ in range(2)] == [8, 0]
    assert slots[:6].tolist() == [(pages - 12) * page] + [3 * page] * 4 + [0] and int(slots[5:].sum()) == 0
    assert cache.held.sum().item() == pages and bool((cache.refs == 1).all())
    assert table[0, :pages - 12].tolist() == [0, 1, 2, *range(15, pages)] and int(table[0, pages - 12]) == -1
    assert int((table >= 0).sum(1)[1:].sum()) == 12
    # and back
    assert int(sg.sage_kv_resize(cache, ints(B)).sum()) == 0 and not bool(cache.refs.any()) and sg.sage_device_status() == 0
