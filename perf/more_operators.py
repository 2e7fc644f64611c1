"""Measured cases of the block-scaled key-value cache and of what a serving program does with its pages.

A case names its operator in ``op``:

  append   new tokens' K and V to an 8-bit cache with one scale for each block of tokens and head
  decode   one new token's attention over that cache
  extend   attention of several new tokens a sequence (a prompt's chunk, drafted tokens) over a cache of
           any kind: 16 bits, 8 bits with a scale a row (``block`` 0) or a block
  fork     a batch that goes on from chosen parents: full pages shared, the page in use copied, pages of
           no sequence freed; then pages for every sequence's next tokens
  compact  the pages in use moved to the front of the pool

``own = False`` computes the operator's plain form from elementary torch operations; ``own = True``
makes the calls of bit_trainable_attention_sage_gb300 that a user's program makes.
"""
import math

import torch

own = False

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
STORE = {"int8": torch.int8, "fp8": torch.float8_e4m3fn}
TOP = {"int8": 127.0, "fp8": 448.0}     # the largest code of the 8-bit formats


def listed():
    return [
        # one decode step: a token of each of 16 sequences goes into the middle of a block
        dict(name="append step", op="append", B=16, Hkv=8, T=1, d=128, dtype="bf16", kind="int8", page=64, block=64, smooth=False),
        # prompts of up to 8192 tokens, ragged, K smoothed, in the blocks that training quantises by
        dict(name="append prompts", op="append", B=4, Hkv=16, T=8192, d=128, dtype="bf16", kind="fp8", page=64, block=64, smooth=True),
        # a ragged serving batch with grouped heads
        dict(name="decode ragged", op="decode", B=16, H=32, Hkv=8, n=4096, even=False, d=128, dtype="bf16", kind="fp8", page=64, block=64),
        # one very long sequence
        dict(name="decode long", op="decode", B=1, H=32, Hkv=8, n=262144, even=True, d=128, dtype="bf16", kind="int8", page=64, block=32),
        # four drafted tokens of each sequence of a ragged batch, verified in one call
        dict(name="extend drafts", op="extend", B=16, H=32, Hkv=8, T=4, n=8192, even=False, d=128, dtype="bf16", kind="int8", page=64, block=64),
        # the next turn of a few conversations: some hundred new tokens, ragged, over a cache with a scale a row
        dict(name="extend turn", op="extend", B=4, H=16, Hkv=4, T=333, n=3000, even=False, d=64, dtype="fp16", kind="fp8", page=16, block=0),
        # a chunk of two long prompts whose earlier chunks are in the cache
        dict(name="extend chunk", op="extend", B=2, H=32, Hkv=8, T=2048, n=6144, even=True, d=128, dtype="bf16", kind="int8", page=64, block=64),
        # the last chunk of a very long prompt, 16-bit pages
        dict(name="extend long", op="extend", B=1, H=16, Hkv=16, T=512, n=65536, even=True, d=128, dtype="bf16", kind="16", page=64, block=0),
        # a step of beam search: 8 prompts of 4 beams each, every beam from one of its prompt's four
        dict(name="fork beams", op="fork", B=32, group=4, n=2000, Hkv=8, d=128, dtype="bf16", kind="fp8", page=64, block=64),
        # 64 answers begun from one long prompt
        dict(name="fork answers", op="fork", B=64, group=64, n=32700, Hkv=8, d=128, dtype="bf16", kind="16", page=128, block=0),
        # a small pool after a few sequences ended
        dict(name="compact few", op="compact", B=8, n=1000, Hkv=8, d=64, dtype="fp16", kind="16", page=16, block=0, ended=3),
        # a large pool of which half the sequences ended
        dict(name="compact half", op="compact", B=32, n=16384, Hkv=8, d=128, dtype="bf16", kind="fp8", page=64, block=64, ended=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "extend", "extend", "fork", "compact"])
    d, dtype = rng.choice([64, 128]), rng.choice(["fp16", "bf16"])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    block = rng.choice([16, 32, 64])
    page = block * rng.choice([k for k in (1, 2, 3, 4) if block * k <= 128])
    kind = rng.choice(["int8", "fp8"])
    c = dict(op=op, Hkv=Hkv, d=d, dtype=dtype, kind=kind, page=page, block=block)
    if op == "append":
        B = rng.randint(1, 16)
        T = max(1, min(_log(rng, 1, 8192), (1 << 22) // (B * Hkv * d // 16)))
        return dict(c, B=B, T=T, smooth=rng.random() < 0.5)
    if op == "decode":
        B = rng.randint(1, 32)
        n = min(_log(rng, 16, 65536), (1 << 28) // (B * Hkv * d))
        return dict(c, B=B, H=Hkv * rng.choice([1, 2, 3, 4, 7, 8, 16]), n=n, even=rng.random() < 0.3)
    if op == "extend":
        c["kind"] = rng.choice(["int8", "int8", "fp8", "fp8", "16"])
        if c["kind"] == "16" or rng.random() < 0.25:
            c["block"] = 0
        B, G = rng.randint(1, 8), rng.choice([1, 2, 3, 4, 7, 8])
        T = max(2, min(_log(rng, 2, 2048), (1 << 17) // (B * Hkv * G)))
        n = min(_log(rng, 1, 32768), (1 << 29) // (B * Hkv * G * T))
        return dict(c, B=B, H=Hkv * G, T=T, n=n, even=rng.random() < 0.4)
    c["kind"] = rng.choice(["fp8", "16"])
    if c["kind"] == "16":
        c["block"] = 0
    if op == "fork":
        group = rng.choice([1, 2, 4, 8])
        B = group * rng.randint(1, 8)
        n = min(_log(rng, 10, 16384), (1 << 27) // (B * Hkv * d))
        return dict(c, B=B, group=group, n=n)
    B = rng.randint(2, 24)
    n = min(_log(rng, 10, 16384), (1 << 28) // (B * Hkv * d))
    return dict(c, B=B, n=n, ended=rng.randint(1, B - 1))


def _lengths(case):
    """The sequences' lengths: all n, or n down to nothing (a batch in mid-flight, an empty row last)."""
    B, n = case["B"], case["n"]
    if B == 1 or case.get("even"):
        return [n] * B
    return [n * (B - 1 - b) // (B - 1) for b in range(B)]


def _counts(case):
    """New tokens of each sequence: all T, or (a ragged batch) T down to T / 2."""
    B, T = case["B"], case["T"]
    return [T] * B if case.get("even") else [T - T * b // (2 * B) for b in range(B)]


def _row_bytes(case):
    """Bytes of a token's K and V of one head, its share of the scales with them."""
    if case["kind"] == "16":
        return 4 * case["d"]
    return 2 * case["d"] + 8 / (case["block"] or 1)


def work(case):
    op, B, Hkv, d, page = case["op"], case["B"], case["Hkv"], case["d"], case["page"]
    row = _row_bytes(case)
    if op == "append":
        rows = Hkv * sum(_counts(case))
        return {"bytes": int(rows * (4 * d + row)), "flops": rows * 2 * d * 4}
    if op == "decode":
        rows, H = Hkv * sum(_lengths(case)), case["H"]
        return {"bytes": int(rows * row) + B * H * (4 * d + 4), "flops": 4 * d * H * sum(_lengths(case))}
    if op == "extend":
        H, lens, counts = case["H"], _lengths(case), _counts(case)
        seen = sum(c * n + c * (c + 1) // 2 for n, c in zip(lens, counts))
        rows = Hkv * sum(n + c for n, c in zip(lens, counts))
        return {"bytes": int(rows * row) + H * sum(counts) * 2 * d + B * H * case["T"] * (2 * d + 4), "flops": 4 * d * H * seen}
    if op == "fork":
        # each group goes on from (about) half its members, or from its one prompt
        lens = _fork_lengths(case)
        copies = sum(lens[b // case["group"] * case["group"]] % page for b in range(B)) // (1 if case["group"] == B else 2)
        entries = sum(-(-n // page) for n in lens)
        return {"bytes": int(2 * copies * Hkv * row) + 12 * entries, "flops": entries}
    lens = _compact_lengths(case)
    need = [-(-n // page) for n in lens]
    left = sum(need) * (B - case["ended"]) // B
    moved = left * (sum(need) - left) // max(1, sum(need))
    return {"bytes": int(2 * moved * Hkv * page * row) + 12 * sum(need), "flops": sum(need)}


def _fork_lengths(case):
    """A group's sequences are equally long; each group is a little shorter than the one before."""
    return [case["n"] - case["n"] * (b // case["group"]) // (2 * case["B"]) for b in range(case["B"])]


def _compact_lengths(case):
    return [case["n"] - case["n"] * b // (2 * case["B"]) for b in range(case["B"])]


# ---- inputs ---------------------------------------------------------------------------------


def _pages(need, g):
    """A page table of scattered pages, -1 behind each sequence's last."""
    total = sum(need)
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(need), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    return table, total


def _store(x, case):
    """A pool's K or V (pages, heads, page, d) in its stored form: codes and scales, or the 16-bit values."""
    kind, block = case["kind"], case["block"]
    if kind == "16":
        return x, None
    s = x.abs().amax(-1).float() / TOP[kind]
    if block:
        s = s.unflatten(-1, (-1, block)).amax(-1)
    y = x.float() / _spread(s, block).unsqueeze(-1)
    return (y.round() if kind == "int8" else y).to(STORE[kind]), s


def _spread(s, block):
    """Scales (pages, heads, page / block) as one a row (pages, heads, page)."""
    return s.repeat_interleave(block, -1) if block else s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, B, Hkv, d, dt, page = case["op"], case["B"], case["Hkv"], case["d"], DT[case["dtype"]], case["page"]
    rand = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=dt)  # noqa: E731
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    st = {"case": case}
    if op in ("fork", "compact"):
        return _prepare_pages(st, case, g, rand, ints)
    counts = [0] * B if op == "decode" else _counts(case)
    # prompts start a sequence; a few tokens follow what is there already
    starts = _lengths(case) if op != "append" else [0 if case["T"] > 64 else 100 + 37 * b for b in range(B)]
    order = torch.randperm(B, generator=g, device="cuda").tolist()
    counts, starts = [counts[i] for i in order], [starts[i] for i in order]
    st["table"], n = _pages([-(-(s + c) // page) for s, c in zip(starts, counts)], g)
    st["pages"] = n
    st["start"], st["count"] = ints(starts), ints(counts)
    shape = (n + 1, Hkv, page, d)                        # one spare page at the pool's end that no table names
    st["cK"], st["sK"] = _store(rand(*shape), case)
    st["cV"], st["sV"] = _store(rand(*shape), case)
    if op == "append":
        st["K"], st["V"] = rand(B, Hkv, case["T"], d), rand(B, Hkv, case["T"], d)
        st["mu"] = None
        if case["smooth"]:
            st["mu"] = torch.randn((B, Hkv, d), generator=g, device="cuda") * 2.0
            st["K"] = (st["K"].float() + st["mu"].unsqueeze(2)).to(dt)
    else:
        st["Q"] = rand(B, case["H"], case.get("T", 1), d)
    return st


def _prepare_pages(st, case, g, rand, ints):
    B, Hkv, d, page = case["B"], case["Hkv"], case["d"], case["page"]
    lens = _fork_lengths(case) if case["op"] == "fork" else _compact_lengths(case)
    need = [-(-n // page) for n in lens]
    if case["op"] == "fork":
        # one prompt for all: only the first sequence has pages; else each its own
        single = case["group"] == B
        if single:
            lens, need = lens[:1] + [0] * (B - 1), need[:1] + [0] * (B - 1)
            parent = [0] * B
        else:
            pick = torch.randint(0, case["group"], (B,), generator=g, device="cuda").tolist()
            parent = [b // case["group"] * case["group"] + pick[b] for b in range(B)]
        table, total = _pages(need, g)
        width = -(-(max(lens) + 1) // page)
        table = torch.cat((table, torch.full((B, 1 + width - table.shape[1]), -1, dtype=torch.int32, device="cuda")), 1)
        pages = total + 2 * B
        spread = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = torch.where(table >= 0, spread[table.long().clamp(min=0)], -1)
        st["parent"], st["lens"] = ints(parent), ints(lens)
    else:
        table, pages = _pages(need, g)
        # sequences that ended left their pages behind
        gone = torch.randperm(B, generator=g, device="cuda")[:case["ended"]].tolist()
        for b in gone:
            table[b] = -1
            need[b] = 0
    shape = (pages + 1, Hkv, page, d)
    st["cK"], st["sK"] = _store(rand(*shape), case)
    st["cV"], st["sV"] = _store(rand(*shape), case)
    st["pages"] = pages
    refs = torch.zeros(pages + 1, dtype=torch.int32, device="cuda")
    refs[table[table >= 0].long()] = 1
    # table, counts of the pages and of each sequence's pages in one buffer, restored before each pass
    st["ints0"] = torch.cat((table.flatten(), refs, ints(need)))
    st["ints"] = st["ints0"].clone()
    t, r, h = st["ints"].split((table.numel(), pages + 1, B))
    st["table"], st["refs"], st["held"] = t.view(table.shape), r[:pages], h
    return st


# ---- one pass -------------------------------------------------------------------------------


def run(st):
    return {"append": _append, "decode": _decode, "extend": _extend, "fork": _fork, "compact": _compact}[st["case"]["op"]](st)


def _cache(st):
    """The framework's handle of the state's cache, made once as a program makes it."""
    import bit_trainable_attention_sage_gb300 as sg
    if "cache" not in st:
        n = st["pages"]
        cut = lambda x: None if x is None else x[:n]  # noqa: E731
        st["cache"] = sg.KvCache(K=cut(st["cK"]), V=cut(st["cV"]), table=st["table"], sK=cut(st["sK"]), sV=cut(st["sV"]),
                                 refs=st.get("refs"), held=st.get("held"))
    return sg, st["cache"]


def _values(st):
    """The pool's contents without the spare page.  E4M3 codes come as E4M3 values beside their scales, INT8
    codes as code * scale."""
    n, block = st["pages"], st["case"]["block"]
    K, V, sK, sV = st["cK"][:n], st["cV"][:n], st["sK"], st["sV"]
    if K.dtype == torch.int8:
        return [K * _spread(sK[:n], block).unsqueeze(-1), V * _spread(sV[:n], block).unsqueeze(-1)]
    return [K, V] + ([] if sK is None else [sK[:n], sV[:n]])


def _append(st):
    c = st["case"]
    if own:
        sg, cache = _cache(st)
        sg.sage_kv_append(cache, st["K"], st["V"], st["start"], count=st["count"], mu=st["mu"])
        return _values(st)
    B, Hkv, T, page, block, spare = c["B"], c["Hkv"], c["T"], c["page"], c["block"], st["pages"]
    t = torch.arange(T, device="cuda")
    h = torch.arange(Hkv, device="cuda")
    start, there = st["start"].long(), t < st["count"].unsqueeze(1)
    slot = start.unsqueeze(1) + t                                                # (B, T)
    table, last = st["table"].long(), st["table"].shape[1] - 1
    at = torch.where(there, table.gather(1, (slot // page).clamp(max=last)), spare)   # the spare page takes what is not there
    where = (at.unsqueeze(1), h.view(1, Hkv, 1), (slot % page).unsqueeze(1))
    blocks = (at.unsqueeze(1), h.view(1, Hkv, 1), (slot % page // block).unsqueeze(1))
    # the block that the first token continues: its rows before that token are kept
    kept = start % block * (st["count"] > 0)
    p0 = torch.where(kept > 0, table.gather(1, (start // page).clamp(max=last).unsqueeze(1)).squeeze(1), spare)
    first = (p0.view(B, 1), h.view(1, Hkv), (start % page // block).view(B, 1))
    rows = (p0.view(B, 1, 1), h.view(1, Hkv, 1), (start % page // block * block).view(B, 1, 1) + torch.arange(block, device="cuda"))
    # a tensor for a divisor: a number's reciprocal would be multiplied by, off by a rounding
    top = torch.full((1,), TOP[c["kind"]], device="cuda")
    for x, pool, scale, mu in ((st["K"], st["cK"], st["sK"], st["mu"]), (st["V"], st["cV"], st["sV"], None)):
        y = x.float() if mu is None else x.float() - mu.unsqueeze(2)
        s = y.abs().amax(-1) / top                                               # (B, Hkv, T)
        flat = ((at.unsqueeze(1) * Hkv + h.view(1, Hkv, 1)) * (page // block) + (slot % page // block).unsqueeze(1)).flatten()
        new = torch.full_like(scale, -1.0).flatten()
        new.scatter_reduce_(0, flat, s.flatten(), "amax")
        old = scale[first]                                                       # (B, Hkv)
        n0 = new.view_as(scale)[first]
        grown = torch.where((kept > 0).unsqueeze(1), torch.maximum(n0, old), n0)
        new = new.view_as(scale)
        new[first] = torch.where((kept > 0).unsqueeze(1), grown, new[first])
        ratio = torch.where(grown > old, old / grown, 1.0)                       # (B, Hkv)
        code = pool.view(torch.int8)[rows].view(pool.dtype).float()              # (B, Hkv, block, d)
        less = code * ratio.view(B, Hkv, 1, 1)
        less = (less.round() if c["kind"] == "int8" else less).to(pool.dtype)
        stays = torch.arange(block, device="cuda") < kept.unsqueeze(1)
        raw = pool.view(torch.int8)
        raw[rows] = torch.where(stays.view(B, 1, block, 1), less.view(torch.int8), raw[rows])
        scale.copy_(torch.where(new >= 0, new, scale))
        s = scale[blocks].unsqueeze(-1)
        y = torch.where(s > 0, y / s, 0.0)
        raw[where] = (y.round() if c["kind"] == "int8" else y).to(pool.dtype).view(torch.int8)
    return _values(st)


def _gathered(pool, scale, st):
    """A pool's pages as (B, Hkv, capacity, d) float32 values."""
    at = st["table"].long().clamp(min=0)
    x = (pool.view(torch.int8)[at].view(pool.dtype) if pool.element_size() == 1 else pool[at]).float()
    if scale is not None:
        x = x * _spread(scale, st["case"]["block"])[at].unsqueeze(-1)
    B, m, H, page, d = x.shape
    return x.transpose(1, 2).reshape(B, H, m * page, d)


def _attention(st, last):
    """Attention over the cache, row (b, t) over the slots up to last[b, t] (-1: none)."""
    c = st["case"]
    B, H, Hkv, d, T = c["B"], c["H"], c["Hkv"], c["d"], st["Q"].shape[2]
    K, V = _gathered(st["cK"], st["sK"], st), _gathered(st["cV"], st["sV"], st)
    out = torch.arange(K.shape[2], device="cuda") > last.unsqueeze(-1)           # (B, T, capacity)
    q = st["Q"].float().view(B, Hkv, H // Hkv * T, d)
    S = (q @ K.transpose(-1, -2)).div_(math.sqrt(d)).view(B, H, T, -1).masked_fill_(out.unsqueeze(1), -math.inf)
    m = S.amax(-1, keepdim=True).clamp(min=-1e30)
    P = S.sub_(m).exp_()
    l = P.sum(-1, keepdim=True)
    O = (P.view(B, Hkv, H // Hkv * T, -1) @ V).view(B, H, T, d) / l.clamp(min=1e-30)
    L = torch.where(last.unsqueeze(1) >= 0, (m + l.log()).squeeze(-1), -math.inf)
    return O.to(st["Q"].dtype), L


def _decode(st):
    if own:
        sg, cache = _cache(st)
        return sg.sage_attn_decode(st["Q"], cache, st["start"])
    return _attention(st, st["start"].unsqueeze(1) - 1)


def _extend(st):
    if own:
        sg, cache = _cache(st)
        return sg.sage_attn_extend(st["Q"], cache, st["start"], count=st["count"])
    t = torch.arange(st["case"]["T"], device="cuda")
    return _attention(st, torch.where(t < st["count"].unsqueeze(1), st["start"].unsqueeze(1) + t, -1))


def _free_pages(st):
    """All pages, the free ones first in ascending order, and their number."""
    used = st["refs"] > 0
    return used.to(torch.int8).sort(stable=True).indices, (~used).sum()


def _fork(st):
    c = st["case"]
    st["ints"].copy_(st["ints0"])           # so that a pass can be run again
    if own:
        sg, cache = _cache(st)
        lens = sg.sage_kv_fork(cache, st["parent"], st["lens"])
        slots = sg.sage_kv_resize(cache, lens + 1)
        return _values(st) + [st["table"], st["refs"], st["held"], lens, slots]
    B, page, P = c["B"], c["page"], st["pages"]
    table, refs, held = st["table"], st["refs"], st["held"]
    M = table.shape[1]
    b, e = torch.arange(B, device="cuda"), torch.arange(M, device="cuda")
    alive, p = st["parent"] >= 0, st["parent"].long().clamp(min=0)
    n = torch.where(alive, st["lens"][p], 0)
    full, part = n // page, n % page
    # a parent's pages in use and in reserve go on with itself or else its first child
    key = torch.where(p == b, -1, b)
    heir = torch.full((B,), B, device="cuda").scatter_reduce_(0, p, torch.where(alive, key, B), "amin")
    heir = alive & (key == heir[p])
    children = torch.zeros(B, dtype=torch.int32, device="cuda").index_add_(0, p, alive.to(torch.int32))
    delta = torch.where(e < (st["lens"] // page).unsqueeze(1), children.unsqueeze(1) - 1, -(children == 0).to(torch.int32).unsqueeze(1))
    delta = torch.where(e < held.unsqueeze(1), delta, 0).to(torch.int32)
    refs.index_add_(0, table.long().clamp(min=0).flatten(), delta.flatten())
    order, free = _free_pages(st)
    need = alive & ~heir & (part > 0)
    rank = need.cumsum(0) - 1
    got = need & (rank < free)
    page_of = torch.where(got, order[rank.clamp(min=0, max=P - 1)], P)
    keep = torch.where(heir, held[p], torch.where(alive, full + got, 0)).to(torch.int32)
    old = table[p]
    src = torch.where(got, old.gather(1, full.long().clamp(max=M - 1).unsqueeze(1)).squeeze(1).long(), P)
    new = torch.where(e == full.unsqueeze(1), torch.where(got, page_of, -1).unsqueeze(1), -1)
    new = torch.where(e < keep.unsqueeze(1), torch.where((e == full.unsqueeze(1)) & ~heir.unsqueeze(1), new, old), -1)
    table.copy_(new)
    refs.index_add_(0, page_of.clamp(max=P - 1), got.to(torch.int32))
    held.copy_(keep)
    stay = torch.arange(page, device="cuda") < part.unsqueeze(1)                 # (B, page)
    for pool in (st["cK"], st["cV"], st["sK"], st["sV"]):
        if pool is not None:
            raw = pool.view(torch.int8) if pool.element_size() == 1 else pool
            step = page // pool.shape[2]                                         # rows a value: 1, or the block
            mask = stay[:, ::step].view(B, 1, -1, *[1] * (pool.dim() - 3))
            raw[page_of] = torch.where(mask, raw[src], raw[page_of])
    lens = torch.where(need & ~got, full * page, n).to(torch.int32)
    return _values(st) + [table, refs, held, lens, _resize(st, lens + 1)]


def _resize(st, want):
    page, P = st["case"]["page"], st["pages"]
    table, refs, held = st["table"], st["refs"], st["held"]
    e = torch.arange(table.shape[1], device="cuda")
    k = -(-want // page)
    drop = (e >= k.unsqueeze(1)) & (e < held.unsqueeze(1))
    refs.index_add_(0, table.long().clamp(min=0).flatten(), -drop.to(torch.int32).flatten())
    order, free = _free_pages(st)
    grow = (k - held).clamp(min=0)
    rank = (grow.cumsum(0) - grow - held).unsqueeze(1) + e
    take = (e >= held.unsqueeze(1)) & (e < k.unsqueeze(1)) & (rank < free)
    page_of = order[rank.clamp(min=0, max=P - 1)]
    refs.index_add_(0, page_of.flatten(), take.to(torch.int32).flatten())
    table.copy_(torch.where(drop, -1, torch.where(take, page_of, table)))
    held.copy_(torch.minimum(held, k) + take.sum(1))
    return held * page


def _compact(st):
    st["ints"].copy_(st["ints0"])
    if own:
        sg, cache = _cache(st)
        used = sg.sage_kv_compact(cache)
        return _values(st) + [st["table"], st["refs"], st["held"], used]
    P, table, refs, held = st["pages"], st["table"], st["refs"], st["held"]
    i = torch.arange(P, device="cuda")
    there = refs > 0
    used = there.sum().to(torch.int32)
    half = max(1, P // 2)
    src = torch.where(there & (i >= used), i, P).sort().values[:half]
    dst = torch.where(~there & (i < used), i, P).sort().values[:half]
    for pool in (st["cK"], st["cV"], st["sK"], st["sV"]):
        if pool is not None:
            raw = pool.view(torch.int8) if pool.element_size() == 1 else pool
            for k in range(0, half, 4096):                   # the spare page goes to itself
                raw[dst[k:k + 4096]] = raw[src[k:k + 4096]]
    to = torch.arange(P + 1, device="cuda").scatter_(0, src, dst)
    count = torch.cat((refs, refs[:1] * 0))
    wide = count.scatter(0, dst, count[src])
    wide = torch.where(torch.arange(P + 1, device="cuda") < used, wide, 0)
    refs.copy_(wide[:P])
    mine = torch.arange(table.shape[1], device="cuda") < held.unsqueeze(1)
    table.copy_(torch.where(mine, to[table.long().clamp(min=0)], table))
    return _values(st) + [table, refs, held, used.view(1)]


# ---- the definition in 64 bits --------------------------------------------------------------


def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _append64, "decode": _decode64, "extend": _extend64, "fork": _fork64, "compact": _compact64}[case["op"]](st, case)


def _stored(pool, scale, block):
    """A pool's values in 64 bits, or its codes beside the scales (E4M3)."""
    return pool.double() if scale is None else pool.double() * _spread(scale, block).double().unsqueeze(-1)


def _append64(st, c):
    """Sequence by sequence, block by block.  A code is a border's matter: the definition names the 32-bit
    values that it is formed from (K - mu, the scale, the quotients), each here the nearest to the 64-bit result."""
    n, page, block = st["pages"], c["page"], c["block"]
    near = lambda v: v.float().double()  # noqa: E731
    code = (lambda v: v.round()) if c["kind"] == "int8" else (lambda v: v.float().to(torch.float8_e4m3fn).double())
    starts, counts, table = st["start"].tolist(), st["count"].tolist(), st["table"].tolist()
    out = []
    for x, pool, scale, mu in ((st["K"], st["cK"], st["sK"], st["mu"]), (st["V"], st["cV"], st["sV"], None)):
        y = x.double() if mu is None else near(x.double() - mu.double().unsqueeze(2))
        codes, scales = pool[:n].double(), scale[:n].double()
        for b, (a, k) in enumerate(zip(starts, counts)):
            t = 0
            while t < k:
                p, off = table[b][(a + t) // page], (a + t) % page
                i, kept = off // block, off % block
                m = min(block - kept, k - t)
                rows = y[b, :, t:t + m]
                s = near(rows.abs().amax((-1, -2)) / TOP[c["kind"]])
                if kept:
                    old = scales[p, :, i].clone()
                    s = torch.maximum(s, old)
                    ratio = torch.where(s > old, near(old / s), 1.0)
                    codes[p, :, off - kept:off] = code(near(codes[p, :, off - kept:off] * ratio.view(-1, 1, 1)))
                scales[p, :, i] = s
                codes[p, :, off:off + m] = code(near(torch.nan_to_num(rows / s.view(-1, 1, 1))))
                t += m
        out.append((codes, scales))
    if c["kind"] == "int8":
        return [k * _spread(s, block).unsqueeze(-1) for k, s in out]
    return [k for k, _ in out] + [s for _, s in out]


def _rows64(st, c, b, h, n):
    """K and V of one head of one sequence, (n, d) in 64 bits."""
    at = st["table"][b, :max(1, -(-n // c["page"]))].long()
    out = []
    for pool, scale in ((st["cK"], st["sK"]), (st["cV"], st["sV"])):
        x = pool[:, h].view(torch.int8)[at].view(pool.dtype) if pool.element_size() == 1 else pool[at, h]
        x = x.double()
        if scale is not None:
            x = (x.unflatten(1, (scale.shape[2], -1)) * scale[at, h].double()[..., None, None]).flatten(1, 2)
        out.append(x.reshape(-1, c["d"])[:n])
    return out


def _decode64(st, c):
    """One sequence and one kv head at a time."""
    B, H, Hkv, d = c["B"], c["H"], c["Hkv"], c["d"]
    G = H // Hkv
    O = torch.zeros((B, H, 1, d), dtype=torch.float64, device="cuda")
    L = torch.full((B, H, 1), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(st["start"].tolist()):
        for h in range(Hkv if n else 0):
            K, V = _rows64(st, c, b, h, n)
            s = st["Q"][b, h * G:(h + 1) * G, 0].double() @ K.T / math.sqrt(d)
            O[b, h * G:(h + 1) * G, 0] = torch.softmax(s, -1) @ V
            L[b, h * G:(h + 1) * G, 0] = torch.logsumexp(s, -1)
    return O, L


def _extend64(st, c):
    """One sequence and one query head at a time, 512 rows at a time."""
    B, H, Hkv, d, T = c["B"], c["H"], c["Hkv"], c["d"], c["T"]
    O = torch.zeros((B, H, T, d), dtype=torch.float64, device="cuda")
    L = torch.full((B, H, T), -math.inf, dtype=torch.float64, device="cuda")
    for b, (a, k) in enumerate(zip(st["start"].tolist(), st["count"].tolist())):
        for h in range(Hkv):
            K, V = _rows64(st, c, b, h, a + k)
            for x in range(h * (H // Hkv), (h + 1) * (H // Hkv)):
                for t in range(0, k, 512):
                    m = min(512, k - t)
                    s = st["Q"][b, x, t:t + m].double() @ K.T / math.sqrt(d)
                    s += torch.full_like(s, -math.inf).triu(a + t + 1)
                    O[b, x, t:t + m] = torch.softmax(s, -1) @ V
                    L[b, x, t:t + m] = torch.logsumexp(s, -1)
    return O, L


def _whole(st, c, K, V, sK, sV):
    n = st["pages"]
    if c["kind"] == "int8":
        return [_stored(K[:n], sK[:n], c["block"]), _stored(V[:n], sV[:n], c["block"])]
    return [K[:n].double(), V[:n].double()] + ([] if sK is None else [sK[:n].double(), sV[:n].double()])


def _fork64(st, c):
    """Sequence by sequence on lists."""
    page, block, B, P = c["page"], c["block"] or 1, c["B"], st["pages"]
    rows, refs, lens, parent = st["table"].tolist(), st["refs"].tolist(), st["lens"].tolist(), st["parent"].tolist()
    M = len(rows[0])
    rows = [r[:k] for r, k in zip(rows, st["held"].tolist())]
    heirs = {}
    for b, p in enumerate(parent):
        if p >= 0 and (p not in heirs or p == b):
            heirs[p] = b
    refs, new, wait = [0] * P, [], []
    for b, p in enumerate(parent):
        full = lens[p] // page if p >= 0 else 0
        new.append([] if p < 0 else list(rows[p]) if heirs[p] == b else rows[p][:full])
        if p >= 0 and heirs[p] != b and lens[p] % page:
            wait.append(b)
    for r in new:
        for x in r:
            refs[x] += 1
    free = [x for x in range(P) if refs[x] == 0]
    out = [lens[p] if p >= 0 else 0 for p in parent]
    K, V, sK, sV = st["cK"], st["cV"], st["sK"], st["sV"]
    for b in wait:
        p, full, part = parent[b], lens[parent[b]] // page, lens[parent[b]] % page
        if not free:
            out[b] = full * page
            continue
        x, y = free.pop(0), rows[p][full]
        new[b].append(x)
        refs[x] = 1
        for pool in (K, V):
            pool.view(torch.uint8)[x, :, :part] = pool.view(torch.uint8)[y, :, :part]
        for s in (sK, sV):
            if s is not None:
                s[x, :, :-(-part // block)] = s[y, :, :-(-part // block)]
    for b in range(B):
        k = -(-(out[b] + 1) // page)
        for x in new[b][k:]:
            refs[x] -= 1
        new[b] = new[b][:k]
    free = [x for x in range(P) if refs[x] == 0]
    for b in range(B):
        while len(new[b]) < -(-(out[b] + 1) // page) and free:
            new[b].append(free.pop(0))
            refs[new[b][-1]] = 1
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    held = [len(r) for r in new]
    return _whole(st, c, K, V, sK, sV) + [ints([r + [-1] * (M - len(r)) for r in new]), ints(refs), ints(held), ints(out), ints([k * page for k in held])]


def _compact64(st, c):
    P, refs, held, rows = st["pages"], st["refs"].tolist(), st["held"].tolist(), st["table"].tolist()
    used = sum(1 for r in refs if r)
    to = dict(zip([x for x in range(used, P) if refs[x]], [x for x in range(used) if not refs[x]]))
    K, V, sK, sV = st["cK"], st["cV"], st["sK"], st["sV"]
    for x, y in to.items():
        refs[x], refs[y] = refs[y], refs[x]
        for pool in (K, V, sK, sV):
            if pool is not None:
                pool.view(torch.uint8)[y] = pool.view(torch.uint8)[x]
    rows = [[to.get(x, x) if i < k else x for i, x in enumerate(r)] for r, k in zip(rows, held)]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    return _whole(st, c, K, V, sK, sV) + [ints(rows), ints(refs), ints(held), ints([used])]
