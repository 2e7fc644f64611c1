"""Plain forms of the cache operators in 64 bits, and caches to test them on."""
from __future__ import annotations

import numpy as np
import torch

KINDS = {"fp16": torch.float16, "bf16": torch.bfloat16, "int8": torch.int8, "fp8": torch.float8_e4m3fn}
U = 2.0 ** -24


def codes_of(x: torch.Tensor, kind: str):
    """(codes, scales) of float32 rows: delta = fl32(max / M), the nearest code of fl32(x / delta), as the
    definition names them (CPU, IEEE float32)."""
    top = torch.full((1,), 127.0 if kind == "int8" else 448.0)
    s = x.abs().amax(-1) / top
    y = torch.where(s.unsqueeze(-1) > 0, x / s.unsqueeze(-1), torch.zeros(()))
    if kind == "int8":
        return y.round().clamp(-127, 127).to(torch.int8), s
    return y.to(torch.float8_e4m3fn), s


def filled(kind, B, H, d, page, lens, *, seed=0, q_dtype=torch.bfloat16, score=False, spare=2, garbage=True, v_scale=1.0,
           shared=()):
    """A cache of scattered pages with contents for `lens`, and its dequantised float64 rows (K, V per sequence).
    Slots past a sequence's end and pages that no sequence owns hold NaN, infinities and the like."""
    import bit_trainable_attention_sage_gb300 as sg
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pages = max(1, sum(need)) + spare
    perm = torch.randperm(pages, generator=g).tolist()
    m = max(1, max(need)) + 1
    # behind a row's last page: numbers that are no pages
    table = torch.randint(-5, 3 * pages, (B, m), generator=g, dtype=torch.int32) * 0 - 7
    at = 0
    for b, k in enumerate(need):
        for i in range(k):
            table[b, i] = perm[at]
            at += 1
    for b, c, k in shared:                      # the first k pages of b are those of c
        table[b, :k] = table[c, :k]
    eight = kind in ("int8", "fp8")
    shape = (pages, H, page, d)
    xs, out = [], []
    for which in range(2):
        x = torch.randn(shape, generator=g) * (v_scale if which else 1.0)
        if eight:
            c, s = codes_of(x, kind)
        else:
            c, s = x.to(KINDS[kind]), None
        xs.append((c, s))
    used = torch.zeros((pages, page), dtype=torch.bool)
    for b, n in enumerate(lens):
        for t in range(n):
            used[table[b, t // page], t % page] = True
    if garbage:
        un = ~used.unsqueeze(1).expand(pages, H, page)
        for c, s in xs:
            if s is not None:
                bad = torch.tensor([float("nan"), float("inf"), -3e38, 0.0])
                s[un] = bad[torch.randint(0, 4, (int(un.sum()),), generator=g)]
                raw = c.view(torch.int8)
                raw[un] = torch.tensor([127, -1, -128, 3], dtype=torch.int8)[torch.randint(0, 4, (int(un.sum()), d), generator=g)]
            else:
                bad = torch.tensor([float("nan"), float("inf"), float("-inf"), torch.finfo(c.dtype).min], dtype=c.dtype)
                c[un] = bad[torch.randint(0, 4, (int(un.sum()), d), generator=g)]
    rows = []
    for c, s in xs:
        v = c.double() if s is None else c.double() * s.double().unsqueeze(-1)
        seqs = []
        for b, n in enumerate(lens):
            idx = torch.arange(n)
            seqs.append(v[table[b, idx // page].long(), :, idx % page].permute(1, 0, 2).numpy())     # (H, n, d)
        rows.append(seqs)
    cap = m * page
    sc = torch.rand((B, H, cap), generator=g) if score else None
    pos = torch.zeros((B, H, cap), dtype=torch.int32) if score else None
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    cache = sg.KvCache(dev(xs[0][0]), dev(xs[1][0]), dev(table), sK=dev(xs[0][1]), sV=dev(xs[1][1]), score=dev(sc), pos=dev(pos))
    return cache, rows[0], rows[1]


def attention64(q, K, V):
    """q (G,d), K, V (n,d) float64 -> O, L, p, and the sizes that the tolerances go by."""
    d = q.shape[-1]
    s = q @ K.T / np.sqrt(d)
    A = np.abs(q) @ np.abs(K).T / np.sqrt(d)
    m = s.max(-1, keepdims=True)
    e = np.exp(s - m)
    l = e.sum(-1, keepdims=True)
    p = e / l
    return p @ V, (m + np.log(l))[:, 0], p, A, p @ np.abs(V)


def tolerances(d, n, A, L):
    """(relative error of a probability, of an output against sum p |v|, absolute error of L).

    A logit is d / 16 tensor-core sums of 16 exact products and the running sum, each term cut at
    2^-24 of the largest or better: 17 u of A = sum |q k| / sqrt(d) a step; the scales (q's and
    log2(e) / sqrt(d) in one, K's) and their product round 3 times.  exp2 and its argument's
    difference add 2^-22 and u (|s - m| log2 e <= 2 A log2 e).  A softmax weight moves by twice the
    largest logit error (itself, and the sum).  Sums of exponentials: a float32 addition a token of
    a lane and a rescaling a granule, n / 32 + 16 roundings of positive terms, and the joins.  The
    second product: n / 64 sums a warp, 17 u each, a rescaling u each, hi + lo 2^-17."""
    a = float(A.max())
    logit = (17 * (d // 16) + 4) * U * a
    weight = 2 * (logit + 2.0 ** -22 + 3 * U * a)
    sums = (n / 32 + 16 + 600) * U      # at most 456 + 4 parts are joined
    prob = weight + 2 * sums
    out = prob + (n / 64 + 8) * 18 * U + 2.0 ** -17
    return prob, out, logit + sums + 2.0 ** -22 + 4 * U * (1 + float(np.abs(L).max()))


def check_decode(Q, O, L, lens, K, V, H, score=None, score0=None):
    """Every output of a decode call against 64 bits."""
    B, Hq, _, d = Q.shape
    G = Hq // H
    q, o, lg = Q.double().cpu().numpy(), O.double().cpu().numpy(), L.double().cpu().numpy()
    eps = torch.finfo(Q.dtype).eps / 2
    tiny = 2.0 ** -25 if Q.dtype == torch.float16 else 2.0 ** -134
    for b, n in enumerate(lens):
        for h in range(H):
            heads = slice(h * G, (h + 1) * G)
            if n == 0:
                assert np.all(o[b, heads] == 0) and np.all(lg[b, heads] == -np.inf)
            else:
                want, Lw, p, A, pv = attention64(q[b, heads, 0], K[b][h], V[b][h])
                prob, out, lse = tolerances(d, n, A, Lw)
                err = np.abs(o[b, heads, 0] - want)
                bound = out * pv + eps * np.abs(want) * (1 + out) + tiny
                assert np.all(err <= bound), (b, h, n, float((err / bound).max()))
                assert np.all(np.abs(lg[b, heads, 0] - Lw) <= lse), (b, h, n, float(np.abs(lg[b, heads, 0] - Lw).max()), lse)
            if score is not None:
                got, was = score[b, h].double().cpu().numpy(), score0[b, h].double().cpu().numpy()
                add = np.zeros_like(was)
                tol = np.zeros_like(was)
                if n:
                    add[:n] = p.sum(0)
                    tol[:n] = (prob + (G + 4) * U) * add[:n] + U * (was[:n] + add[:n]) * 1.01 + 1e-37
                assert np.all(np.abs(got - (was + add)) <= tol), (b, h, n)


def evict64(score, pos, n, seen, budget, recent):
    """Slots of one row: (destinations, sources) of the moves, by sorting."""
    if n <= budget:
        return [], []
    key = []
    for s in range(n):
        x = float(score[s])
        fresh = int(pos[s]) >= seen - recent
        key.append(((0, 0.0) if fresh else (2, 0.0) if x != x else (1, -x), s))
    stay = sorted(s for _, s in sorted(key)[:budget])
    kept = set(stay)
    return [s for s in range(budget) if s not in kept], [s for s in stay if s >= budget]
