"""Plain forms of the block-scaled cache on the CPU (IEEE float32), and caches to test it on."""
from __future__ import annotations

import torch

STORE = {"int8": torch.int8, "fp8": torch.float8_e4m3fn}
TOP = {"int8": 127.0, "fp8": 448.0}


def quotients(x, s, kind):
    """The nearest codes of fl32(x / s), 0 where s is 0, as float32 values."""
    y = torch.where(s > 0, x / s, torch.zeros(()))
    if kind == "int8":
        return y.round().clamp(-127, 127)
    return y.clamp(-448, 448).to(torch.float8_e4m3fn).float()


def append_blocks(pool, scale, table, x, start, count, block, kind):
    """x (B,H,T,d) float32 rows to slots start[b] + t of pool (pages,H,page,d) codes as float32 values and scale
    (pages,H,page/block), in place, block by block as the definition says."""
    page = pool.shape[2]
    top = torch.full((1,), TOP[kind])
    for b, (a, n) in enumerate(zip(start, count)):
        t = 0
        while t < n:
            p, off = int(table[b, (a + t) // page]), (a + t) % page
            i, kept = off // block, off % block
            m = min(block - kept, n - t)
            rows = x[b, :, t:t + m]
            s = rows.abs().amax((-1, -2)) / top
            if kept:
                old = scale[p, :, i].clone()
                s = torch.maximum(s, old)
                grown = (s > old).view(-1, 1, 1)
                ratio = torch.where(s > old, old / s, torch.ones(())).view(-1, 1, 1)
                was = pool[p, :, off - kept:off]
                less = was * ratio
                less = less.round() if kind == "int8" else less.clamp(-448, 448).to(torch.float8_e4m3fn).float()
                pool[p, :, off - kept:off] = torch.where(grown, less, was)
            scale[p, :, i] = s
            pool[p, :, off:off + m] = quotients(rows, s.view(-1, 1, 1), kind)
            t += m


def filled_blocks(kind, B, H, d, page, block, lens, *, seed=0, spare=2, room=0, v_scale=1.0, garbage=True, shared=()):
    """A block-scaled cache of scattered pages with contents for ``lens`` (pages for ``room`` more tokens), and its
    dequantised float64 rows (K, V per sequence, (H, n, d)).  Blocks of no row hold garbage codes and scales, rows
    behind a sequence's end in its last block garbage codes."""
    import bit_trainable_attention_sage_gb300 as sg
    g = torch.Generator().manual_seed(seed)
    need = [-(-(n + room) // page) for n in lens]
    pages = max(1, sum(need)) + spare
    perm = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((B, max(1, max(need)) + 1), -7, dtype=torch.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = perm[at:at + k]
        at += k
    for b, c, k in shared:                      # the first k pages of b are those of c
        table[b, :k] = table[c, :k]
    used = torch.zeros((pages, page), dtype=torch.bool)
    for b, n in enumerate(lens):
        for t in range(n):
            used[table[b, t // page], t % page] = True
    blocks = used.view(pages, page // block, block).any(-1)
    out, rows = [], []
    for which in range(2):
        x = torch.randn((pages, H, page, d), generator=g) * (v_scale if which else 1.0)
        # scales of several sizes, so that a wrong block's shows
        x *= torch.exp2(torch.randint(-3, 4, (pages, H, page // block), generator=g).float()).repeat_interleave(block, -1).unsqueeze(-1)
        s = x.abs().amax(-1).unflatten(-1, (-1, block)).amax(-1) / torch.full((1,), TOP[kind])
        c = quotients(x, s.repeat_interleave(block, -1).unsqueeze(-1), kind).to(STORE[kind])
        if garbage:
            un = ~used.unsqueeze(1).expand(pages, H, page)
            raw = c.view(torch.int8)
            raw[un] = torch.tensor([127, -1, -128, 3], dtype=torch.int8)[torch.randint(0, 4, (int(un.sum()), d), generator=g)]
            no = ~blocks.unsqueeze(1).expand(pages, H, page // block)
            s[no] = torch.tensor([float("nan"), float("inf"), -3e38, 0.0])[torch.randint(0, 4, (int(no.sum()),), generator=g)]
        out.append((c, s))
        v = c.double() * s.double().repeat_interleave(block, -1).unsqueeze(-1)
        rows.append([v[table[b, torch.arange(n) // page].long(), :, torch.arange(n) % page].permute(1, 0, 2).numpy() for b, n in enumerate(lens)])
    (K, sK), (V, sV) = out
    cache = sg.KvCache(K.cuda(), V.cuda(), table.cuda(), sK=sK.cuda(), sV=sV.cuda())
    return cache, rows[0], rows[1]
