"""Pages of a pool that sequences share: given, taken back, forked and compacted, against the rules on lists."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "int8": torch.int8, "fp8": torch.float8_e4m3fn}


def _sg():
    import bit_trainable_attention_sage_gb300 as sg
    return sg


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def raw(t):
    return t.view({1: torch.int8, 2: torch.int16, 4: torch.int32}[t.element_size()])


class Model:
    """The same cache on lists: each row's pages, the pool's tensors on the CPU."""

    def __init__(self, cache):
        self.page, self.P, self.B, self.M, self.block = cache.page, cache.pages, cache.B, cache.table.shape[1], cache.block or 1
        self.rows = [[] for _ in range(self.B)]
        self.pools = [raw(t).cpu().clone() for t in (cache.K, cache.V)]
        self.scales = [raw(t).cpu().clone() for t in (cache.sK, cache.sV) if t is not None]
        self.short = False

    def free(self):
        used = {p for r in self.rows for p in r}
        return [p for p in range(self.P) if p not in used]

    def resize(self, want):
        need = [-(-w // self.page) for w in want]
        for r, k in zip(self.rows, need):
            del r[k:]
        free = self.free()
        for r, k in zip(self.rows, need):
            while len(r) < k:
                if not free:
                    self.short = True
                    break
                r.append(free.pop(0))
        return [len(r) * self.page for r in self.rows]

    def fork(self, parent, lens):
        was = [list(r) for r in self.rows]
        heir = {}
        for b, p in enumerate(parent):
            if p >= 0 and (p not in heir or p == b):
                heir[p] = b
        out, copy = [], []
        for b, p in enumerate(parent):
            if p < 0:
                self.rows[b] = []
            elif heir[p] == b:
                self.rows[b] = list(was[p])
            else:
                self.rows[b] = was[p][:lens[p] // self.page]
                if lens[p] % self.page:
                    copy.append(b)
            out.append(lens[p] if p >= 0 else 0)
        free = self.free()
        for b in copy:
            p = parent[b]
            full, part = divmod(lens[p], self.page)
            if not free:
                self.short = True
                out[b] = full * self.page
                continue
            dst, src = free.pop(0), was[p][full]
            self.rows[b].append(dst)
            for t in self.pools:
                t[dst, :, :part] = t[src, :, :part]
            for t in self.scales:
                t[dst, :, :-(-part // self.block)] = t[src, :, :-(-part // self.block)]
        return out

    def compact(self):
        used = sorted({p for r in self.rows for p in r})
        U = len(used)
        to = dict(zip([p for p in used if p >= U], [p for p in range(U) if p not in set(used)]))
        for src, dst in to.items():
            for t in self.pools + self.scales:
                t[dst] = t[src]
        self.rows = [[to.get(p, p) for p in r] for r in self.rows]
        return U

    def check(self, cache):
        table, refs = cache.table.tolist(), [0] * self.P
        for b, r in enumerate(self.rows):
            assert table[b] == r + [-1] * (self.M - len(r)), b
            for p in r:
                refs[p] += 1
        assert cache.held.tolist() == [len(r) for r in self.rows] and cache.refs.tolist() == refs
        for t, want in zip((cache.K, cache.V), self.pools):
            assert torch.equal(raw(t).cpu(), want)
        for t, want in zip((cache.sK, cache.sV), self.scales):
            assert torch.equal(raw(t).cpu(), want)


def pool(kind, B, H, d, page, pages, max_pages, block=0, seed=0):
    sg = _sg()
    cache = sg.make_kv_cache(B, H, d, page * max_pages, dtype=DT[kind], page=page, block=block, pages=pages)
    g = torch.Generator(device="cuda").manual_seed(seed)
    for t in (cache.K, cache.V, cache.sK, cache.sV):
        if t is not None:
            r = raw(t)
            r.copy_(torch.randint(-100, 100, r.shape, generator=g, device="cuda"))
    return cache, Model(cache)


@pytest.mark.parametrize("kind,d,page,block,pages", [("int8", 128, 64, 64, 40), ("fp8", 64, 48, 16, 40), ("fp16", 64, 16, 0, 40), ("int8", 64, 32, 0, 40),
                                                     ("bf16", 128, 128, 0, 40), ("fp8", 128, 96, 32, 40), ("int8", 64, 32, 16, 13)])
def test_many_calls(kind, d, page, block, pages):
    """A mixture of all three, with sequences that end, grow, shrink and share; the smallest pool runs out of pages."""
    sg = _sg()
    rng = random.Random(page + d)
    B, M = 9, 7
    cache, model = pool(kind, B, 3, d, page, pages, M, block)
    lens, short = [0] * B, False
    for step in range(40):
        what = rng.choice(["resize", "resize", "fork", "compact"])
        model.short = False
        if what == "resize":
            want = [rng.choice([0, 1, page, page + 1, rng.randint(0, M * page), len(model.rows[b]) * page, M * page]) for b in range(B)]
            slots = sg.sage_kv_resize(cache, ints(want))
            assert slots.tolist() == model.resize(want)
            lens = [rng.randint(0, s) if rng.random() < 0.8 else s for s in slots.tolist()]
        elif what == "fork":
            parent = [rng.choice([-1, b, rng.randrange(B), rng.randrange(B)]) for b in range(B)]
            if step % 9 == 0:
                parent = [rng.randrange(B)] * B
            out = sg.sage_kv_fork(cache, ints(parent), ints(lens))
            assert out.tolist() == model.fork(parent, lens)
            lens = out.tolist()
        else:
            assert sg.sage_kv_compact(cache).tolist() == [model.compact()]
        assert sg.sage_device_status() == (8 if model.short else 0), what
        short = short or model.short
        model.check(cache)
    assert short or pages > 13


def test_many_sequences_and_pages():
    """More sequences and pages than a plan has threads."""
    sg = _sg()
    rng = random.Random(1)
    B, page, M = 5000, 16, 40
    cache, model = pool("int8", B, 1, 64, page, 90000, M, 16)
    want = [rng.choice([0, 1, rng.randint(0, 600)]) for _ in range(B)]
    assert sg.sage_kv_resize(cache, ints(want)).tolist() == model.resize(want)
    parent = [rng.choice([-1, b, rng.randrange(B)]) for b in range(B)]
    assert sg.sage_kv_fork(cache, ints(parent), ints(want)).tolist() == (lens := model.fork(parent, want))
    model.check(cache)
    want = [n + 1 if rng.random() < 0.5 else 0 for n in lens]
    assert sg.sage_kv_resize(cache, ints(want)).tolist() == model.resize(want)
    assert sg.sage_kv_compact(cache).tolist() == [model.compact()]
    model.check(cache)
    assert sg.sage_device_status() == 0


def test_compact_at_its_ends():
    """An empty pool, a full one, one in use at its front and one at its back."""
    sg = _sg()
    cache, model = pool("fp8", 4, 2, 64, 16, 12, 12, 16)
    for want in ([0] * 4, [16, 16, 16, 16], [16 * 3] * 4, [0, 0, 0, 16 * 3], [0] * 4, [16 * 12, 0, 0, 0], [16, 0, 0, 0]):
        assert sg.sage_kv_resize(cache, ints(want)).tolist() == model.resize(want)
        assert sg.sage_kv_compact(cache).tolist() == [model.compact()]
        model.check(cache)
    assert sg.sage_device_status() == 0


def test_one_page_and_one_sequence():
    sg = _sg()
    cache, model = pool("fp16", 1, 1, 64, 16, 1, 1)
    for want in ([1], [16], [0], [7]):
        assert sg.sage_kv_resize(cache, ints(want)).tolist() == model.resize(want)
    assert sg.sage_kv_fork(cache, ints([0]), ints([7])).tolist() == [7]
    assert sg.sage_kv_compact(cache).tolist() == [1]
    assert sg.sage_kv_fork(cache, ints([-1]), ints([7])).tolist() == [0]
    model.rows = [[]]
    model.check(cache)


def test_inputs_out_of_range():
    """Held to their range, or left alone, and reported; nothing outside the cache is touched."""
    sg = _sg()
    cache, model = pool("int8", 4, 2, 64, 16, 20, 5, 16)
    assert sg.sage_kv_resize(cache, ints([33, -5, 1 << 30, 1])).tolist() == model.resize([33, 0, 80, 1])
    assert sg.sage_device_status() == 7
    model.check(cache)
    # a parent that is none: the sequence itself; lengths past what a sequence holds: all of it
    assert sg.sage_kv_fork(cache, ints([4, 2, -2, 0]), ints([33, 5, 99, 1])).tolist() == model.fork([0, 2, 2, 0], [33, 0, 80, 1])
    assert sg.sage_device_status() == 7
    model.check(cache)
    # a table entry that is no page: nothing moves, so that nothing looks at it; then it stays, whatever else moves
    cache.table[0, 1] = 77
    sg.sage_kv_compact(cache)
    assert int(cache.table[0, 1]) == 77 and sg.sage_device_status() == 0
    last = int(cache.table[2, 4])
    cache.table[2, 4] = 19
    cache.refs[19], cache.refs[last] = cache.refs[last].clone(), 0
    cache.table[1, 4] = 19
    used = int(sg.sage_kv_compact(cache))
    assert int(cache.table[0, 1]) == 77 and sg.sage_device_status() == 7
    assert cache.table[1:3, 4].tolist() == [last, last] and used == int((cache.refs > 0).sum()) > last
    cache.held[1] = 9
    sg.sage_kv_resize(cache, ints([0, 0, 0, 0]))
    assert sg.sage_device_status() == 7 and cache.held.tolist() == [0] * 4
    # an entry that names a page of no count
    cache, model = pool("int8", 2, 1, 64, 16, 8, 2, 16)
    cache.table[0, 0], cache.table[1, 0] = 6, 7
    cache.held.fill_(1)
    cache.refs[7] = 1
    assert sg.sage_kv_compact(cache).tolist() == [1] and sg.sage_device_status() == 7
    assert cache.table[:, 0].tolist() == [6, 0]


def test_status_words_are_kept_apart():
    sg = _sg()
    cache, _ = pool("int8", 2, 1, 64, 16, 3, 8, 16)
    sg.sage_kv_resize(cache, ints([16 * 5, -1]))
    assert [sg.sage_device_status() for _ in range(3)] == [7, 8, 0]
    assert "free page" in sg.sage_status_string(8)


def test_binding_refuses():
    sg = _sg()
    cache = sg.make_kv_cache(2, 1, 64, 64, pages=5, score=True)
    two, three = ints([0, 0]), ints([0, 0, 0])
    with pytest.raises(ValueError, match="cannot be shared"):
        sg.sage_kv_fork(cache, two, two)
    with pytest.raises(ValueError, match="shape"):
        sg.sage_kv_resize(cache, three)
    with pytest.raises(TypeError):
        sg.sage_kv_resize(cache, two.long())
    with pytest.raises(ValueError, match="refs and held"):
        sg.sage_kv_compact(sg.make_kv_cache(2, 1, 64, 64))
    with pytest.raises(ValueError, match="workspace"):
        sg.sage_kv_compact(cache, workspace=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(sg.SageError):
        sg.sage_kv_compact(cache, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(sg.SageError):
        sg.sage_kv_resize(cache, two, out=two)
    K = torch.zeros(4, 1, 16, 64, dtype=torch.half, device="cuda")
    table = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="belong together"):
        sg.KvCache(K, K.clone(), table, refs=ints([0] * 4))
    with pytest.raises(ValueError, match="refs"):
        sg.KvCache(K, K.clone(), table, refs=ints([0] * 3), held=ints([0]))


@pytest.mark.parametrize("stream", [False, True])
def test_beams(stream):
    """A beam search of several steps (fork, resize, append, decode) answers as caches that copy everything do; every
    call on the current stream, or all of them captured once and replayed on another."""
    sg = _sg()
    B, H, Hq, d, page = 6, 2, 4, 64, 16
    steps, n0 = 25, 37
    K0, V0 = (torch.randn(1, H, n0, d, device="cuda").bfloat16() for _ in range(2))
    pool_ = sg.make_kv_cache(B, H, d, 128, dtype=torch.int8, page=page, block=16, pages=40)
    alone = sg.make_kv_cache(B, H, d, 128, dtype=torch.int8, page=page, block=16)
    lens = ints([n0] + [0] * (B - 1))
    sg.sage_kv_resize(pool_, lens)
    first = torch.zeros(B, H, n0, d, dtype=torch.bfloat16, device="cuda")
    K, V = first.clone(), first.clone()
    K[0], V[0] = K0[0], V0[0]
    sg.sage_kv_append(pool_, K, V, ints([0] * B), count=ints([n0] + [0] * (B - 1)))
    for b in range(B):
        K[b], V[b] = K0[0], V0[0]
    sg.sage_kv_append(alone, K, V, ints([0] * B))
    at = torch.full((B,), n0, dtype=torch.int32, device="cuda")
    parent = ints([0] * B)
    k, v = (torch.zeros(B, H, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros(B, Hq, 1, d, dtype=torch.bfloat16, device="cuda")
    one = ints([1] * B)

    def shared():
        new = sg.sage_kv_fork(pool_, parent, lens)
        sg.sage_kv_resize(pool_, new + one)
        sg.sage_kv_append(pool_, k, v, new)
        lens.copy_(new + one)
        return sg.sage_attn_decode(q, pool_, lens)
    state = [t.clone() for t in (pool_.table, pool_.refs, pool_.held, lens, pool_.K, pool_.V, pool_.sK, pool_.sV)]
    if stream:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = shared()
        for t, s in zip((pool_.table, pool_.refs, pool_.held, lens, pool_.K, pool_.V, pool_.sK, pool_.sV), state):
            t.copy_(s)
    for step in range(steps):
        for t in (k, v, q):
            t.normal_()
        if step:
            parent.copy_(torch.randint(0, B, (B,), device="cuda", dtype=torch.int32))
            own = alone.table.long()
            for t in (alone.K, alone.V, alone.sK, alone.sV):
                r = raw(t)
                r[own] = r[own[parent.long()]].clone()
        if stream:
            graph.replay()
        else:
            out = shared()
        sg.sage_kv_append(alone, k, v, at)
        at += one
        O, L = sg.sage_attn_decode(q, alone, at)
        assert torch.equal(lens, at) and torch.equal(out[0], O) and torch.equal(out[1], L), step
    assert sg.sage_device_status() == 0
    rows = [pool_.table[b, :int(pool_.held[b])].tolist() for b in range(B)]
    assert len({p for r in rows for p in r}) < sum(len(r) for r in rows)      # they do share
    used = sg.sage_kv_compact(pool_)
    O, L = sg.sage_attn_decode(q, pool_, lens)
    assert torch.equal(out[0], O) and torch.equal(out[1], L)
    assert int(pool_.table.max()) < int(used) == int((pool_.refs > 0).sum())


def test_another_stream():
    sg = _sg()
    cache, model = pool("int8", 3, 2, 64, 16, 20, 5, 16)
    s = torch.cuda.Stream()
    want = ints([40, 1, 17])
    s.wait_stream(torch.cuda.current_stream())
    slots = sg.sage_kv_resize(cache, want, stream=s)
    lens = sg.sage_kv_fork(cache, ints([0, 0, 2]), want, stream=s)
    sg.sage_kv_compact(cache, stream=s)
    s.synchronize()
    assert slots.tolist() == model.resize([40, 1, 17]) and lens.tolist() == model.fork([0, 0, 2], [40, 1, 17])
    model.compact()
    model.check(cache)


def test_a_shared_pool_with_scores():
    """Resize and compact beside scores: rows of scores are the sequences' own, and eviction goes on as before."""
    sg = _sg()
    B, H, d = 3, 2, 64
    cache = sg.make_kv_cache(B, H, d, 128, dtype=torch.int8, page=16, score=True, pages=30)
    alone = sg.make_kv_cache(B, H, d, 128, dtype=torch.int8, page=16, score=True)
    lens = ints([100, 33, 64])
    assert sg.sage_kv_resize(cache, lens).tolist() == [112, 48, 64]
    assert sg.sage_kv_resize(cache, ints([100, 0, 64])).tolist() == [112, 0, 64]
    assert int(sg.sage_kv_compact(cache)) == 11 and sg.sage_kv_resize(cache, lens).tolist() == [112, 48, 64]
    k, v = (torch.randn(B, H, 100, d).bfloat16().cuda() for _ in range(2))
    q = torch.randn(B, 4, 1, d).bfloat16().cuda()
    for c in (cache, alone):
        sg.sage_kv_append(c, k, v, ints([0] * B), count=lens)
    out = [(*sg.sage_attn_decode(q, c, lens, score=True), sg.sage_kv_evict(c, lens, lens, budget=40, recent=8)) for c in (cache, alone)]
    assert all(torch.equal(a, b) for a, b in zip(*out)) and torch.equal(cache.score, alone.score) and torch.equal(cache.pos, alone.pos)
    assert sg.sage_kv_resize(cache, out[0][2]).tolist() == [48, 48, 48] and int(sg.sage_kv_compact(cache)) == 9
    a, b = (sg.sage_attn_decode(q, c, out[0][2]) for c in (cache, alone))
    assert torch.equal(a[0], b[0]) and sg.sage_device_status() == 0
