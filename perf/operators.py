"""Measured cases of the serving operators: rotary positions, the paged key-value cache, attention
of one new token over it, and eviction from it.

A case names its operator in ``op``:

  rope    multi-axis rotary positions of Q and K (``inverse``: the gradient's direction)
  append  new tokens' K and V written to the pages of a cache (16-bit, INT8 or E4M3)
  decode  one new token's attention over the cache (``score``: accumulates the weights)
  evict   the cache cut to ``budget`` tokens by accumulated weight

``own = False`` computes the operator's plain form from elementary torch operations; ``own = True``
makes the calls of bit_trainable_attention_sage_gb300 that a user's program makes.
"""
import math

import torch

own = False

DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
STORE = {"int8": torch.int8, "fp8": torch.float8_e4m3fn}
TOP = {"int8": 127.0, "fp8": 448.0}     # the largest code of the 8-bit formats
BASE = 10000.0


def listed():
    return [
        # one decode step of a batch of 16: the new tokens' queries and keys, image/text positions
        dict(name="rope step", op="rope", B=16, H=32, Hkv=8, N=1, d=128, dtype="bf16", axes=3, interleaved=False, inverse=False, far=1 << 20),
        # the headline training shape, positions of a video (time, height, width)
        dict(name="rope train", op="rope", B=2, H=16, Hkv=16, N=8192, d=128, dtype="fp16", axes=3, interleaved=False, inverse=False, far=8192),
        # the gradient of the 4096-token training shape: float32, as the attention backward gives it
        dict(name="rope grad", op="rope", B=4, H=16, Hkv=16, N=4096, d=128, dtype="fp32", axes=1, interleaved=True, inverse=True, far=4096),
        # one decode step: a token of each of 16 sequences goes to the cache in its own type
        dict(name="append step", op="append", B=16, Hkv=8, T=1, d=128, dtype="bf16", kind="16", page=64, smooth=False),
        # prompts of up to 8192 tokens, ragged, K smoothed, stored as E4M3
        dict(name="append prompts", op="append", B=4, Hkv=16, T=8192, d=128, dtype="bf16", kind="fp8", page=64, smooth=True),
        # a single short sequence: latency
        dict(name="decode one", op="decode", B=1, H=8, Hkv=8, n=1000, even=True, d=64, dtype="fp16", kind="16", page=64, score=False),
        # a ragged serving batch with grouped heads over INT8 pages, weights accumulated for eviction
        dict(name="decode ragged int8", op="decode", B=16, H=32, Hkv=8, n=4096, even=False, d=128, dtype="bf16", kind="int8", page=64, score=True),
        # a full batch at the headline's length, one kv head a query head
        dict(name="decode batch", op="decode", B=32, H=16, Hkv=16, n=8191, even=True, d=128, dtype="bf16", kind="16", page=64, score=False),
        # one very long sequence, grouped heads, E4M3 pages of 16 tokens
        dict(name="decode long fp8", op="decode", B=1, H=32, Hkv=8, n=262144, even=True, d=128, dtype="bf16", kind="fp8", page=16, score=False),
        # two long sequences, d = 64, weights accumulated
        dict(name="decode scored", op="decode", B=2, H=32, Hkv=4, n=32768, even=True, d=64, dtype="fp16", kind="16", page=128, score=True),
        # steady state: every 64 steps the cache is cut back to 1024 tokens a head
        dict(name="evict step", op="evict", B=8, Hkv=8, n=1088, even=True, budget=1024, recent=128, d=128, dtype="bf16", kind="16", page=64),
        # long prompts cut to a quarter after prefill
        dict(name="evict prompts", op="evict", B=4, Hkv=8, n=32768, even=False, budget=8192, recent=1024, d=128, dtype="bf16", kind="fp8", page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "decode", "decode", "evict"])
    d = rng.choice([64, 128])
    dtype = rng.choice(["fp16", "bf16"])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    if op == "rope":
        B, G = rng.randint(1, 16), rng.choice([1, 2, 4])
        N = _log(rng, 1, 8192)
        N = max(1, min(N, (1 << 21) // (B * Hkv * (1 + G) * d // 8)))
        return dict(op=op, B=B, H=Hkv * G, Hkv=Hkv, N=N, d=d, dtype=rng.choice([dtype, dtype, "fp32"]), axes=rng.randint(1, 3), interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5, far=_log(rng, 64, 1 << 20))
    page = rng.choice([16, 32, 48, 64, 128])
    kind = rng.choice(["16", "int8", "fp8"])
    if op == "append":
        B = rng.randint(1, 16)
        T = min(_log(rng, 1, 8192), (1 << 22) // (B * Hkv * d // 16))
        return dict(op=op, B=B, Hkv=Hkv, T=T, d=d, dtype=dtype, kind=kind, page=page, smooth=kind != "16" and rng.random() < 0.5)
    B = rng.randint(1, 32)
    if op == "decode":
        G = rng.choice([1, 2, 3, 4, 7, 8, 16])
        n = min(_log(rng, 16, 65536), (1 << 28) // (B * Hkv * d))
        return dict(op=op, B=B, H=Hkv * G, Hkv=Hkv, n=n, even=rng.random() < 0.3, d=d, dtype=dtype, kind=kind, page=page, score=rng.random() < 0.4)
    kind = rng.choice(["16", "fp8"])
    n = min(_log(rng, 128, 32768), (1 << 26) // (B * Hkv * d))
    budget = max(16, int(n * rng.uniform(0.2, 0.95)))
    return dict(op=op, B=B, Hkv=Hkv, n=n, even=rng.random() < 0.5, budget=budget, recent=int(budget * rng.uniform(0, 0.5)), d=d, dtype=dtype, kind=kind, page=page)


def _lengths(case):
    """The sequences' lengths: all n, or n down to nothing (a batch in mid-flight, an empty row last)."""
    B, n = case["B"], case["n"]
    if case["even"] or B == 1:
        return [n] * B
    return [n * (B - 1 - b) // (B - 1) for b in range(B)]


def _counts(case):
    """New tokens of each sequence: all T, or (a prompt batch) T down to T / 2."""
    B, T = case["B"], case["T"]
    return [T - T * b // (2 * B) for b in range(B)]


def _sections(case):
    """Pairs of each axis: a quarter for time and three eighths each for height and width."""
    half = case["d"] // 2
    return {1: (half,), 2: (half // 2, half // 2), 3: (half // 4, half * 3 // 8, half * 3 // 8)}[case["axes"]]


def _bytes_of(case):
    return 2 if case["kind"] == "16" else 1


def work(case):
    op, B, d = case["op"], case["B"], case["d"]
    if op == "rope":
        n = B * (case["H"] + case["Hkv"]) * case["N"] * d
        return {"bytes": 2 * n * (4 if case["dtype"] == "fp32" else 2) + 4 * case["axes"] * B * case["N"], "flops": 3 * n}
    es, Hkv = _bytes_of(case), case["Hkv"]
    scales = 0 if es == 2 else 8
    if op == "append":
        rows = Hkv * sum(_counts(case))
        return {"bytes": rows * (2 * d * (2 + es) + scales), "flops": rows * 2 * d * (4 if es == 1 else 1)}
    lens = _lengths(case)
    if op == "decode":
        rows, H = Hkv * sum(lens), case["H"]
        return {"bytes": rows * (2 * d * es + scales + (8 if case["score"] else 0)) + B * H * (4 * d + 4), "flops": 4 * d * H * sum(lens)}
    budget, recent = case["budget"], case["recent"]
    moved = sum(Hkv * budget * (1 - (budget - recent) / max(1, n - recent)) for n in lens if n > budget)
    return {"bytes": 8 * Hkv * sum(n for n in lens if n > budget) + moved * 2 * (2 * d * es + scales + 8), "flops": Hkv * sum(lens)}


# ---- inputs ---------------------------------------------------------------------------------


def _pages(lens, page, g):
    """A pool with a page table of scattered pages, -1 behind each sequence's last; one spare page at the
    pool's end that no table names."""
    need = [-(-n // page) for n in lens]
    total = sum(need)
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    return table, total


def _store(x, kind):
    """A pool's K or V in its stored form: codes and one scale a token, or the 16-bit values."""
    if kind == "16":
        return x, None
    s = x.abs().amax(-1).float() / TOP[kind]
    y = x.float() / s.unsqueeze(-1)
    return (y.round() if kind == "int8" else y).to(STORE[kind]), s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, B, d, dt = case["op"], case["B"], case["d"], DT[case["dtype"]]
    rand = lambda *s, t=dt, v=1.0: (torch.randn(s, generator=g, device="cuda", dtype=t if t != torch.float32 else None) * v)  # noqa: E731
    st = {"case": case}
    if op == "rope":
        N, v = case["N"], 1e-2 if case["inverse"] else 1.0
        st["Q"], st["K"] = rand(B, case["H"], N, d, v=v), rand(B, case["Hkv"], N, d, v=v)
        # runs of consecutive positions that start anywhere up to `far`, on every axis
        first = torch.randint(0, max(1, case["far"] - N + 1), (case["axes"], B, 1), generator=g, device="cuda")
        st["positions"] = (first + torch.arange(N, device="cuda")).to(torch.int32)
        half = d // 2
        st["freqs"] = [BASE ** (-j / half) for j in range(half)]
        st["sections"] = _sections(case)
        return st
    Hkv, page, kind = case["Hkv"], case["page"], case["kind"]
    if op == "append":
        counts = _counts(case)
        order = torch.randperm(B, generator=g, device="cuda").tolist()
        counts = [counts[i] for i in order]
        # prompts start a sequence; a single token follows what is there already
        starts = [0 if case["T"] > 1 else 100 + 37 * i for i in order]
        st["table"], st["pages"] = _pages([s + c for s, c in zip(starts, counts)], page, g)
        st["start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        st["count"] = torch.tensor(counts, dtype=torch.int32, device="cuda")
        st["K"], st["V"] = rand(B, Hkv, case["T"], d), rand(B, Hkv, case["T"], d)
        st["mu"] = None
        if case["smooth"]:
            st["mu"] = rand(B, Hkv, d, t=torch.float32, v=2.0)
            st["K"] = (st["K"].float() + st["mu"].unsqueeze(2)).to(dt)
        shape = (st["pages"] + 1, Hkv, page, d)
        st["cK"], st["cV"] = (torch.zeros(shape, dtype=dt if kind == "16" else STORE[kind], device="cuda") for _ in range(2))
        st["sK"], st["sV"] = (None if kind == "16" else torch.zeros(shape[:3], device="cuda") for _ in range(2))
        return st
    lens = _lengths(case)
    order = torch.randperm(B, generator=g, device="cuda").tolist()
    lens = [lens[i] for i in order]
    st["table"], st["pages"] = _pages(lens, page, g)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    shape = (st["pages"] + 1, Hkv, page, d)
    st["cK"], st["sK"] = _store(rand(*shape), kind)
    st["cV"], st["sV"] = _store(rand(*shape), kind)
    cap = st["table"].shape[1] * page
    st["score0"] = torch.empty((B, Hkv, cap), device="cuda").exponential_(generator=g)
    st["score"] = st["score0"].clone()
    if op == "decode":
        st["Q"] = rand(B, case["H"], 1, d)
        return st
    # every token's position in the text: what earlier evictions left, then the recent ones
    seen, recent = 2 * case["n"], case["recent"]
    old = torch.rand((B, Hkv, seen - recent), generator=g, device="cuda").argsort(-1)
    pos = torch.zeros((B, Hkv, cap), dtype=torch.int32, device="cuda")
    for b, n in enumerate(lens):
        k = max(0, n - recent)
        pos[b, :, :k] = old[b, :, :k].to(torch.int32)
        pos[b, :, k:n] = torch.arange(seen - (n - k), seen, dtype=torch.int32, device="cuda")
    st["pos0"], st["pos"] = pos, pos.clone()
    st["seen"] = torch.full((B,), seen, dtype=torch.int32, device="cuda")
    return st


# ---- one pass -------------------------------------------------------------------------------


def run(st):
    return {"rope": _rope, "append": _append, "decode": _decode, "evict": _evict}[st["case"]["op"]](st)


def _cache(st):
    """The framework's handle of the state's cache, made once as a program makes it."""
    import bit_trainable_attention_sage_gb300 as sg
    if "cache" not in st:
        st["cache"] = sg.KvCache(K=st["cK"], V=st["cV"], table=st["table"], sK=st.get("sK"), sV=st.get("sV"), score=st.get("score"), pos=st.get("pos"))
    return sg, st["cache"]


def _values(st):
    """The cache's contents without the spare page.  E4M3 codes come as E4M3 values beside their scales,
    INT8 codes as code * scale."""
    n = st["pages"]
    K, V, sK, sV = st["cK"][:n], st["cV"][:n], st["sK"], st["sV"]
    if K.dtype == torch.int8:
        return [K * sK[:n].unsqueeze(-1), V * sV[:n].unsqueeze(-1)]
    return [K, V] + ([] if sK is None else [sK[:n], sV[:n]])


def _rope(st):
    c = st["case"]
    if own:
        import bit_trainable_attention_sage_gb300 as sg
        if "rope" not in st:
            st["rope"] = sg.make_rope(c["d"], st["sections"], base=BASE, interleaved=c["interleaved"])
        return sg.sage_rope(st["Q"], st["K"], st["positions"], st["rope"], inverse=c["inverse"])
    # angles in 64 bits: far positions lose their last turns in 32
    f = torch.tensor(st["freqs"], dtype=torch.float64, device="cuda")
    axis = torch.repeat_interleave(torch.arange(c["axes"], device="cuda"), torch.tensor(st["sections"], device="cuda"), output_size=c["d"] // 2)
    angle = st["positions"][axis].permute(1, 2, 0).double() * f                 # (B, N, d/2)
    cos, sin = angle.cos().float().unsqueeze(1), angle.sin().float().unsqueeze(1)
    if c["inverse"]:
        sin = -sin
    return tuple(_rotated(st[k], cos, sin, c["interleaved"]) for k in ("Q", "K"))


def _rotated(x, cos, sin, interleaved):
    y = x.float()
    x0, x1 = (y[..., 0::2], y[..., 1::2]) if interleaved else y.chunk(2, -1)
    y0, y1 = x0 * cos - x1 * sin, x0 * sin + x1 * cos
    return (torch.stack((y0, y1), -1).flatten(-2) if interleaved else torch.cat((y0, y1), -1)).to(x.dtype)


def _append(st):
    c = st["case"]
    if own:
        sg, cache = _cache(st)
        sg.sage_kv_append(cache, st["K"], st["V"], st["start"], count=st["count"], mu=st["mu"])
        return _values(st)
    B, Hkv, T, page = c["B"], c["Hkv"], c["T"], c["page"]
    t = torch.arange(T, device="cuda")
    slot = st["start"].long().unsqueeze(1) + t                                   # (B, T)
    at = st["table"].long().gather(1, (slot // page).clamp(max=st["table"].shape[1] - 1))
    at = torch.where(t < st["count"].unsqueeze(1), at, st["pages"])              # the spare page takes what is not there
    where = (at.unsqueeze(1), torch.arange(Hkv, device="cuda").view(1, Hkv, 1), (slot % page).unsqueeze(1))
    for x, pool, scale, mu in ((st["K"], st["cK"], st["sK"], st["mu"]), (st["V"], st["cV"], st["sV"], None)):
        if scale is None:
            pool[where] = x
            continue
        y = x.float() if mu is None else x.float() - mu.unsqueeze(2)
        # a tensor for a divisor: a number's reciprocal would be multiplied by, off by a rounding
        s = y.abs().amax(-1) / torch.full((1,), TOP[c["kind"]], device="cuda")
        y = torch.where(s.unsqueeze(-1) > 0, y / s.unsqueeze(-1), 0.0)
        y = (y.round() if c["kind"] == "int8" else y).to(pool.dtype)
        pool.view(torch.int8)[where] = y.view(torch.int8)
        scale[where] = s
    return _values(st)


def _gathered(pool, scale, table, dtype):
    """A pool's pages as (B, Hkv, capacity, d) values."""
    at = table.long().clamp(min=0)
    x = (pool.view(torch.int8)[at].view(pool.dtype) if pool.element_size() == 1 else pool[at]).to(dtype)
    if scale is not None:
        x = x * scale[at].unsqueeze(-1)
    B, m, H, page, d = x.shape
    return x.transpose(1, 2).reshape(B, H, m * page, d)


def _decode(st):
    c = st["case"]
    B, H, Hkv, d = c["B"], c["H"], c["Hkv"], c["d"]
    if c["score"]:
        st["score"].copy_(st["score0"])     # so that a pass can be run again
    if own:
        sg, cache = _cache(st)
        O, L = sg.sage_attn_decode(st["Q"], cache, st["lens"], score=c["score"])
        return (O, L, st["score"]) if c["score"] else (O, L)
    K = _gathered(st["cK"], st["sK"], st["table"], torch.float32)
    V = _gathered(st["cV"], st["sV"], st["table"], torch.float32)
    out = (torch.arange(K.shape[2], device="cuda") >= st["lens"].unsqueeze(1)).view(B, 1, 1, -1)
    q = st["Q"].float().view(B, Hkv, H // Hkv, d)
    S = (q @ K.transpose(-1, -2) / math.sqrt(d)).masked_fill_(out, -math.inf)
    m = S.amax(-1, keepdim=True).clamp(min=-1e30)
    P = (S - m).exp()
    l = P.sum(-1, keepdim=True)
    P = P / l.clamp(min=1e-30)
    O = (P @ V).to(st["Q"].dtype).view(B, H, 1, d)
    L = (m + l.log()).view(B, H, 1)
    L = torch.where(st["lens"].view(B, 1, 1) > 0, L, -math.inf)
    if c["score"]:
        st["score"] += P.sum(2)
        return O, L, st["score"]
    return O, L


def _evict(st):
    c = st["case"]
    budget, recent, page = c["budget"], c["recent"], c["page"]
    st["score"].copy_(st["score0"])         # so that a pass can be run again: the moved rows' sources stay
    st["pos"].copy_(st["pos0"])
    if own:
        sg, cache = _cache(st)
        lens = sg.sage_kv_evict(cache, st["lens"], st["seen"], budget=budget, recent=recent)
        return _values(st) + [st["score"], st["pos"], lens]
    B, Hkv, cap = st["score"].shape
    slot = torch.arange(cap, device="cuda")
    there = (slot < st["lens"].unsqueeze(1)).unsqueeze(1)                        # (B, 1, cap)
    key = st["score"].masked_fill(st["pos"] >= (st["seen"] - recent).view(B, 1, 1), math.inf)
    key = key.masked_fill(~there, -math.inf)
    rank = key.sort(dim=-1, descending=True, stable=True).indices
    stays = torch.zeros_like(key, dtype=torch.bool).scatter_(-1, rank[..., :budget], True) & there
    free, move = ~stays & there & (slot < budget), stays & (slot >= budget)
    # the i-th freed slot takes the i-th row that moves; what has no partner goes from and to the spare page
    pairs = min(budget, max(1, cap - budget))
    dst, src = (_first(x, pairs) for x in (free, move))
    none = src >= cap
    b, h = torch.arange(B, device="cuda").view(B, 1, 1), torch.arange(Hkv, device="cuda").view(1, Hkv, 1)
    last = cap - 1
    page_of = lambda s: torch.where(none, st["pages"], st["table"].long()[b, s.clamp(max=last) // page])  # noqa: E731
    to, of = (page_of(dst), h, dst % page), (page_of(src), h, src % page)
    for pool in (st["cK"], st["cV"], st["sK"], st["sV"]):
        if pool is not None:
            raw = pool.view(torch.int8) if pool.element_size() == 1 else pool
            raw[to] = raw[of]
    for x in (st["score"], st["pos"]):
        wide = torch.cat((x, x[..., :1]), -1)
        wide.scatter_(-1, torch.where(none, cap, dst), wide.gather(-1, torch.where(none, cap, src)))
        x.copy_(wide[..., :cap])
    return _values(st) + [st["score"], st["pos"], st["lens"].clamp(max=budget)]


def _first(mask, k):
    """The slots of the first k true places of each row, in order; the row's length where there are fewer."""
    cap = mask.shape[-1]
    slot = torch.arange(cap, device=mask.device)
    at = torch.where(mask, slot, cap)
    return at.sort(dim=-1).values[..., :k]


# ---- the definition in 64 bits --------------------------------------------------------------


def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": _rope64, "append": _append64, "decode": _decode64, "evict": _evict64}[case["op"]](st, case)


def _rope64(st, c):
    """x0 + i x1 times e^(i angle), the pairs as complex numbers."""
    half = c["d"] // 2
    angle = torch.empty((c["B"], 1, c["N"], half), dtype=torch.float64, device="cuda")
    j = 0
    for a, pairs in enumerate(st["sections"]):
        for _ in range(pairs):
            angle[:, 0, :, j] = st["positions"][a].double() * st["freqs"][j]
            j += 1
    turn = torch.polar(torch.ones_like(angle), -angle if c["inverse"] else angle)
    out = []
    for x in (st["Q"], st["K"]):
        y = x.double()
        if c["interleaved"]:
            out.append(torch.view_as_real(torch.view_as_complex(y.unflatten(-1, (half, 2)).contiguous()) * turn).flatten(-2))
        else:
            z = torch.complex(y[..., :half].contiguous(), y[..., half:].contiguous()) * turn
            out.append(torch.cat((z.real, z.imag), -1))
    return tuple(out)


def _append64(st, c):
    """Sequence by sequence, page by page.  A code is a border's matter: the definition names the 32-bit values
    that it is formed from (K - mu, the scale, the quotient), each here the nearest to the 64-bit result."""
    n, page = st["pages"], c["page"]
    near = lambda v: v.float().double()  # noqa: E731
    pools = []
    for x, mu in ((st["K"], st["mu"]), (st["V"], None)):
        y = x.double() if mu is None else near(x.double() - mu.double().unsqueeze(2))
        s = near(y.abs().amax(-1) / TOP.get(c["kind"], 1.0))
        pool = torch.zeros((n, c["Hkv"], page, c["d"]), dtype=torch.float64, device="cuda")
        scale = torch.zeros((n, c["Hkv"], page), dtype=torch.float64, device="cuda")
        if c["kind"] != "16":
            # a code is the nearest of the format's values, ties to even
            y = near(torch.nan_to_num(y / s.unsqueeze(-1)))
            y = y.round() if c["kind"] == "int8" else y.float().to(torch.float8_e4m3fn).double()
        for b, (a, k) in enumerate(zip(st["start"].tolist(), st["count"].tolist())):
            t = 0
            while t < k:
                off = (a + t) % page
                m = min(page - off, k - t)
                p = int(st["table"][b, (a + t) // page])
                pool[p, :, off:off + m] = y[b, :, t:t + m]
                scale[p, :, off:off + m] = s[b, :, t:t + m]
                t += m
        pools.append((pool, scale))
    if c["kind"] == "int8":
        return [p * s.unsqueeze(-1) for p, s in pools]
    return [p for p, _ in pools] + ([] if c["kind"] == "16" else [s for _, s in pools])


def _decode64(st, c):
    """One sequence and one kv head at a time."""
    B, H, Hkv, d, page = c["B"], c["H"], c["Hkv"], c["d"], c["page"]
    G = H // Hkv
    O = torch.zeros((B, H, 1, d), dtype=torch.float64, device="cuda")
    L = torch.full((B, H, 1), -math.inf, dtype=torch.float64, device="cuda")
    score = st["score0"].double()
    for b, n in enumerate(st["lens"].tolist()):
        if n == 0:
            continue
        at = st["table"][b, :-(-n // page)].long()
        for h in range(Hkv):
            rows = []
            for pool, scale in ((st["cK"], st["sK"]), (st["cV"], st["sV"])):
                x = pool[:, h].view(torch.int8)[at].view(pool.dtype) if pool.element_size() == 1 else pool[at, h]
                x = x.reshape(-1, d)[:n].double()
                rows.append(x if scale is None else x * scale[at, h].reshape(-1)[:n].double().unsqueeze(-1))
            s = st["Q"][b, h * G:(h + 1) * G, 0].double() @ rows[0].T / math.sqrt(d)
            p = torch.softmax(s, -1)
            O[b, h * G:(h + 1) * G, 0] = p @ rows[1]
            L[b, h * G:(h + 1) * G, 0] = torch.logsumexp(s, -1)
            score[b, h, :n] += p.sum(0)
    return (O, L, score) if c["score"] else (O, L)


def _evict64(st, c):
    """Row by row: the tokens in the order of their rank, then the moves."""
    budget, recent, page = c["budget"], c["recent"], c["page"]
    B, Hkv, cap = st["score0"].shape
    score, pos, lens = st["score0"].double(), st["pos0"].clone(), st["lens"].tolist()
    pools = [None if x is None else x.view(torch.int8) if x.element_size() == 1 else x for x in (st["cK"], st["cV"], st["sK"], st["sV"])]
    for b, n in enumerate(lens):
        for h in range(Hkv):
            if n <= budget:
                continue
            fresh = pos[b, h, :n] >= int(st["seen"][b]) - recent
            worth = torch.where(fresh, math.inf, score[b, h, :n])
            stay = (-worth).sort(stable=True).indices[:budget].sort().values
            src = stay[stay >= budget]
            gone = torch.ones(budget, dtype=torch.bool, device="cuda")
            gone[stay[stay < budget]] = False
            dst = gone.nonzero().flatten()
            row = st["table"][b].long()
            for x in pools:
                if x is not None:
                    x[row[dst // page], h, dst % page] = x[row[src // page], h, src % page]
            score[b, h, dst], pos[b, h, dst] = score[b, h, src], pos[b, h, src]
    n = st["pages"]
    K, V = st["cK"][:n].double(), st["cV"][:n].double()
    scales = [] if st["sK"] is None else [st["sK"][:n].double(), st["sV"][:n].double()]
    return [K, V] + scales + [score, pos, torch.tensor([min(x, budget) for x in lens], dtype=torch.int32, device="cuda")]
