"""Thin ctypes binding of the position and cache calls of libsage_gb300.so (include/sage.h):
rotary positions, the paged key-value cache, attention of one or several new tokens over it, eviction,
and the pages of a pool that sequences share.

As in binding.py, every function has the name of the C entry point it wraps, checks and marshals
its arguments, and takes outputs and workspaces from PyTorch; nothing is computed here.  Calls run
on ``stream`` or else on the current stream of the tensors' device; what a call allocates belongs
to that stream.  Lengths, page tables and positions are device int32 and are not read by the host:
a page, length or slot out of range is skipped and reported by sage_device_status().
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from .binding import SAGE_BF16, SAGE_FP16, _check, _ptr, _workspace, lib

SAGE_FP32 = 2
SAGE_KV_16, SAGE_KV_INT8, SAGE_KV_FP8 = 0, 1, 2
KV_BLOCKS = (16, 32, 64)            # rows that may share a scale
_KINDS = {torch.float16: SAGE_KV_16, torch.bfloat16: SAGE_KV_16, torch.int8: SAGE_KV_INT8,
          torch.float8_e4m3fn: SAGE_KV_FP8}
_DTYPES = {torch.float16: SAGE_FP16, torch.bfloat16: SAGE_BF16, torch.float32: SAGE_FP32}


class SageKv(ctypes.Structure):
    """struct sage_kv (include/sage.h)."""
    _fields_ = [(n, ctypes.c_int) for n in ("B", "H", "d", "dtype", "kind", "page", "pages", "max_pages")] + \
               [(n, ctypes.c_void_p) for n in ("K", "V", "sK", "sV", "table", "score", "pos")]


class SageRopeParams(ctypes.Structure):
    """struct sage_rope_params (include/sage.h)."""
    _fields_ = [(n, ctypes.c_int) for n in ("B", "H", "Hk", "N", "d", "dtype", "axes", "pos_batch", "rotary",
                                            "interleaved", "inverse")] + \
               [("sections", ctypes.POINTER(ctypes.c_int)), ("freq", ctypes.POINTER(ctypes.c_double))]


def _need(t: torch.Tensor, what: str, dtype, shape, device):
    """A contiguous tensor of this type and shape on this device."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == device.index and t.is_contiguous():
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a tensor, got {type(t).__name__}")
    if t.dtype is not dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{what}: must be a contiguous tensor on {device}")


def _workspace_ok(ws, device):
    if ws is not None and (ws.device != device or not ws.is_contiguous()):
        raise ValueError(f"workspace: must be a contiguous tensor on {device}")


def _cuda(device):
    if device.type != "cuda":
        raise ValueError(f"SageBwd tensors must be CUDA tensors, these are on {device}")


def _elsewhere(stream, device) -> bool:
    """Whether the call has to change the current stream or device first (with _on).
    torch.cuda.current_device() would check that CUDA is initialised; the call's tensors show it."""
    return stream is not None or torch._C._cuda_getDevice() != device.index


@contextlib.contextmanager
def _on(stream, device):
    """Makes ``stream`` (or the device's current stream) current, so that the launch and what is
    allocated for it belong to the same stream and device."""
    if stream is None:
        with torch.cuda.device(device):
            yield
    elif stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
    else:
        with torch.cuda.stream(stream):
            yield


def _current(device) -> int:
    """Handle of the device's current stream.  torch.cuda.current_stream() builds an object for it
    (3 us on the GB300's host cores, as long as a launch); this returns the handle alone (0.1 us)."""
    return torch._C._cuda_getCurrentRawStream(device.index)


# ---- rotary positions -----------------------------------------------------------------------


class Rope:
    """What a rotation is besides its positions: made once by make_rope."""

    def __init__(self, d: int, sections, freqs, interleaved: bool):
        self.d, self.sections, self.freqs, self.interleaved = d, tuple(sections), tuple(freqs), bool(interleaved)
        self.axes, self.rotary = len(self.sections), 2 * sum(self.sections)
        self._sections = (ctypes.c_int * self.axes)(*self.sections)
        self._freq = (ctypes.c_double * len(self.freqs))(*self.freqs)
        self._made = {}         # params structs by what they depend on

    def __reduce__(self):
        return Rope, (self.d, self.sections, self.freqs, self.interleaved)   # structs and arrays are made again

    def _struct(self, *key):
        """The struct for (B, H, Hk, N, dtype, pos_batch, inverse)."""
        p = self._made.get(key)
        if p is None:
            if len(self._made) >= 64:
                self._made = {}
            B, H, Hk, N, dtype, pb, inverse = key
            p = self._made[key] = ctypes.byref(SageRopeParams(B, H, Hk, N, self.d, _DTYPES[dtype], self.axes, pb, self.rotary,
                                                              self.interleaved, inverse, self._sections, self._freq))
        return p


def make_rope(d: int, sections, *, base: float = 10000.0, interleaved: bool = False, freqs=None) -> Rope:
    """Rotary positions of heads of ``d`` channels: ``sections[a]`` pairs turn by axis a's position,
    sum(sections) = rotary / 2 <= d / 2 pairs in all (a multiple of 8; channels behind them pass
    through).  Pair j turns by base^(-2j / rotary) radians a position, or by ``freqs[j]``."""
    sections = [int(s) for s in sections]
    pairs = sum(sections)
    if d not in (64, 128):
        raise ValueError(f"d must be 64 or 128, got {d}")
    if not 1 <= len(sections) <= 8 or min(sections) < 0 or pairs % 8 or not 8 <= pairs <= d // 2:
        raise ValueError(f"sections {tuple(sections)}: 1 to 8 axes whose pairs add up to a multiple of 8, at most d / 2")
    if freqs is None:
        if not 0 < base < float("inf"):
            raise ValueError(f"base must be positive, got {base}")
        freqs = [float(base) ** (-j / pairs) for j in range(pairs)]
    freqs = [float(f) for f in freqs]
    if len(freqs) != pairs or not all(abs(f) <= 1e15 for f in freqs):
        raise ValueError(f"freqs: expected {pairs} finite values, one for each pair")
    return Rope(d, sections, freqs, interleaved)


def sage_rope(Q: torch.Tensor, K: torch.Tensor | None, positions: torch.Tensor, rope: Rope, *, inverse: bool = False,
              out=None, stream=None):
    """Rotary positions of Q (B,H,N,d) and K (B,Hk,N,d, or None), fp16, bf16 or float32.
    ``positions`` (axes,B,N) int32, or (axes,1,N) for every sequence the same.  ``inverse`` turns
    back: the gradient.  ``out`` (Qo, Ko) may be (Q, K).  Returns (Qo, Ko)."""
    shape, dtype, dev = Q.shape, Q.dtype, Q.device
    B, H, N, d = shape
    if dtype not in _DTYPES:
        raise TypeError(f"sage_rope takes fp16, bf16 or float32 tensors, got {dtype}")
    _cuda(dev)
    _need(Q, "Q", dtype, shape, dev)
    if d != rope.d:
        raise ValueError(f"Q has {d} channels, the rope {rope.d}")
    Hk = 0
    if K is not None:
        Hk = K.shape[1]
        _need(K, "K", dtype, (B, Hk, N, d), dev)
    pb = 1 if positions.dim() == 3 and positions.shape[1] == 1 else B
    _need(positions, "positions", torch.int32, (rope.axes, pb, N), dev)
    if _elsewhere(stream, dev):
        with _on(stream, dev):
            return sage_rope(Q, K, positions, rope, inverse=inverse, out=out)
    if out is None:
        Qo, Ko = torch.empty_like(Q), None if K is None else torch.empty_like(K)
    else:
        Qo, Ko = out
        _need(Qo, "out[0]", dtype, shape, dev)
        if K is not None:
            _need(Ko, "out[1]", dtype, K.shape, dev)
    st = lib().sage_rope(rope._struct(B, H, Hk, N, dtype, pb, bool(inverse)), Q.data_ptr(), None if K is None else K.data_ptr(),
                         positions.data_ptr(), Qo.data_ptr(), None if K is None else Ko.data_ptr(), _current(dev))
    _check("sage_rope", st)
    return Qo, Ko


# ---- paged key-value cache ------------------------------------------------------------------


def _kv_sizes(B: int, H: int, d: int, page: int, pages: int, max_pages: int, block: int = 0):
    """The sizes that struct sage_kv takes."""
    if min(B, H, page, pages, max_pages) < 1:
        raise ValueError(f"a cache of {B} sequences, {H} heads, {pages} pages of {page} tokens, {max_pages} a sequence: none may be 0")
    if d not in (64, 128):
        raise ValueError(f"d must be 64 or 128, got {d}")
    if page % 16:
        raise ValueError(f"page must be a multiple of 16 tokens, got {page}")
    if max_pages * page >= 1 << 30:
        raise ValueError(f"{max_pages} pages of {page} tokens a sequence: fewer than 2^30 slots are wanted")
    if B * H > 65535:
        raise ValueError(f"{B} sequences of {H} heads: at most 65535 rows are taken")
    if block and (block not in KV_BLOCKS or page % block):
        raise ValueError(f"block must be 16, 32 or 64 rows and divide the page of {page}, got {block}")


class KvCache:
    """A paged key-value cache over tensors of the caller (struct sage_kv).

    K, V (pages,H,page,d): fp16 or bf16 values, or int8 / float8_e4m3fn codes with sK, sV
    (pages,H,page) float32, one scale a row, or (pages,H,page/R), one for each block of R = 16, 32 or 64
    rows; page a multiple of 16, B * H at most 65535.  table (B,max_pages) int32: the pages of each
    sequence; entries behind its last page are not read.  score (B,H,max_pages*page) float32 and
    pos (same, int32) are there for sage_attn_decode(score=True) and sage_kv_evict (not with scales of
    blocks).  refs (pages) and held (B) int32, both or none, are there for a pool that sequences share
    (sage_kv_resize, sage_kv_fork, sage_kv_compact): how many table entries name each page, and how many of each
    row's entries are its pages; these calls write them and table, by a workspace that the object holds (calls that are
    captured into a graph take theirs from the graph's memory, so that a graph can outlive the object).  The tensors are
    fixed for the life of the object; their contents are the caller's and the calls'."""

    def __init__(self, K: torch.Tensor, V: torch.Tensor, table: torch.Tensor, *, sK=None, sV=None, score=None, pos=None, refs=None,
                 held=None):
        if K.dtype not in _KINDS or K.dim() != 4 or table.dim() != 2:
            raise ValueError("K must be (pages,H,page,d) in fp16, bf16, int8 or float8_e4m3fn, table (B,max_pages)")
        pages, H, page, d = K.shape
        B, max_pages = table.shape
        dev = K.device
        block = page // sK.shape[2] if isinstance(sK, torch.Tensor) and sK.dim() == 3 and 0 < sK.shape[2] < page else 0
        _kv_sizes(B, H, d, page, pages, max_pages, block)
        _cuda(dev)
        _need(K, "K", K.dtype, K.shape, dev)
        _need(V, "V", K.dtype, K.shape, dev)
        _need(table, "table", torch.int32, table.shape, dev)
        self.kind = _KINDS[K.dtype]
        if (self.kind == SAGE_KV_16) != (sK is None) or (sK is None) != (sV is None):
            raise ValueError("sK and sV belong to int8 and float8_e4m3fn pools, and only to them")
        for name, t in (("sK", sK), ("sV", sV)):
            if t is not None:
                _need(t, name, torch.float32, (pages, H, page // (block or 1)), dev)
        if block and (score is not None or pos is not None):
            raise ValueError("a cache with scales of blocks has no score and no pos: rows are not evicted from it")
        self.block = block
        self.capacity = max_pages * page
        for name, t, dt in (("score", score, torch.float32), ("pos", pos, torch.int32)):
            if t is not None:
                _need(t, name, dt, (B, H, self.capacity), dev)
        if (refs is None) != (held is None):
            raise ValueError("refs and held belong together")
        if refs is not None:
            _need(refs, "refs", torch.int32, (pages,), dev)
            _need(held, "held", torch.int32, (B,), dev)
        self.K, self.V, self.sK, self.sV, self.table, self.score, self.pos = K, V, sK, sV, table, score, pos
        self.refs, self.held = refs, held
        self.B, self.H, self.d, self.page, self.pages, self.device = B, H, d, page, pages, dev
        # a struct for each 16-bit type that calls may bring
        types = (K.dtype,) if self.kind == SAGE_KV_16 else (torch.float16, torch.bfloat16)
        self._c = {t: ctypes.byref(SageKv(B, H, d, _DTYPES[t], self.kind | block << 8, page, pages, max_pages, K.data_ptr(), V.data_ptr(),
                                          _ptr(sK), _ptr(sV), table.data_ptr(), _ptr(score), _ptr(pos))) for t in types}
        self._bytes = {}        # workspace sizes by what they depend on
        # the page calls' workspace: they all write table, refs and held, so that no two may run at once anyway
        # (with what every such call passes, looked up once: their time is mostly the host's)
        self._any = next(iter(self._c.values()))
        self._pages = None
        if refs is not None:
            ws = self._pages_ws = _workspace(lib().sage_pages_workspace_bytes(self._any), dev)
            self._pages = refs.data_ptr(), held.data_ptr(), (ws.data_ptr(), ws.numel())
            self._pages_streams = {_current(dev)}       # that the allocator knows to use the workspace

    def _struct(self, t: torch.Tensor, what: str):
        """The struct for a call on 16-bit tensors like ``t``."""
        c = self._c.get(t.dtype)
        if c is None:
            raise TypeError(f"{what}: the cache takes {', '.join(map(str, self._c))}, got {t.dtype}")
        return c


def make_kv_cache(B: int, H: int, d: int, capacity: int, *, dtype=torch.int8, page: int = 64, score: bool = False,
                  block: int = 0, pages: int | None = None, device="cuda") -> KvCache:
    """A cache for B sequences of up to ``capacity`` tokens, each with pages of its own; ``score``
    adds what eviction needs.  dtype: fp16, bf16, int8 or float8_e4m3fn.  ``block`` (8-bit types): one
    scale for each block of 16, 32 or 64 rows instead of one a row.  ``pages``: a pool of so many pages that the
    sequences share, all free; sage_kv_resize gives them out."""
    device = torch.device(device)
    if device.type == "cuda" and device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    m = max(1, -(-capacity // max(page, 1)))
    shared = pages is not None
    pages = B * m if pages is None else pages
    _kv_sizes(B, H, d, page, pages, m, block)
    eight = dtype in (torch.int8, torch.float8_e4m3fn)
    if block and (score or not eight):
        raise ValueError("block belongs to int8 and float8_e4m3fn caches without score")
    ints = lambda n, v: torch.full((n,), v, dtype=torch.int32, device=device)  # noqa: E731
    table = ints(B * m, -1).view(B, m) if shared else torch.arange(B * m, dtype=torch.int32, device=device).view(B, m)
    shape = (pages, H, page, d)
    K, V = (torch.zeros(shape, dtype=dtype, device=device) for _ in range(2))
    sK, sV = (torch.zeros((pages, H, page // (block or 1)), device=device) if eight else None for _ in range(2))
    extra = [torch.zeros((B, H, m * page), dtype=t, device=device) if score else None for t in (torch.float32, torch.int32)]
    return KvCache(K, V, table, sK=sK, sV=sV, score=extra[0], pos=extra[1], refs=ints(pages, 0) if shared else None,
                   held=ints(B, 0) if shared else None)


def sage_kv_append(cache: KvCache, K: torch.Tensor, V: torch.Tensor, start: torch.Tensor, *, count=None, mu=None,
                   pos=None, stream=None) -> None:
    """Writes tokens 0 .. count[b] - 1 (None: all T) of K, V (B,H,T,d) to slots start[b] + t of the
    cache, in its form.  ``mu`` (B,H,d) float32 (8-bit caches): K-smoothing, codes of K - mu.
    ``pos`` (B) int32: position in the text of each sequence's first new token (None: its slot).
    With scales of blocks a block's scale grows with its rows (the codes before start[b] follow), and
    what it holds behind the last new token is lost.  It does not shrink when tokens are taken back (a start
    below an earlier call's end), until a call begins the block anew.
    Scores of the new slots are 0: decoding adds to them, weights of a prompt's own queries are the
    caller's to write to cache.score."""
    shape, dev = K.shape, cache.device
    B, H, T, d = shape
    c = cache._struct(K, "K")
    _need(K, "K", K.dtype, (cache.B, cache.H, T, cache.d), dev)
    _need(V, "V", K.dtype, shape, dev)
    _need(start, "start", torch.int32, (B,), dev)
    if count is not None:
        _need(count, "count", torch.int32, (B,), dev)
    if mu is not None:
        _need(mu, "mu", torch.float32, (B, H, d), dev)
    if pos is not None:
        _need(pos, "pos", torch.int32, (B,), dev)
    if _elsewhere(stream, dev):
        with _on(stream, dev):
            return sage_kv_append(cache, K, V, start, count=count, mu=mu, pos=pos)
    st = lib().sage_kv_append(c, K.data_ptr(), V.data_ptr(), T, start.data_ptr(), _ptr(count), _ptr(mu), _ptr(pos), _current(dev))
    _check("sage_kv_append", st)


def sage_attn_decode(Q: torch.Tensor, cache: KvCache, lens: torch.Tensor, *, score: bool = False, out=None, lse=None,
                     workspace=None, stream=None):
    """Attention of one new token a sequence, Q (B,Hq,1,d), over its lens[b] cached slots; Hq is a
    multiple of the cache's heads.  ``score`` adds the attention weights to cache.score.  A ``workspace``
    of the caller's begins at a multiple of 256 bytes, as PyTorch's allocations do.
    Returns (O (B,Hq,1,d) in Q's type, L (B,Hq,1) float32); a sequence of no slots gives 0 and -inf."""
    shape, dtype, dev = Q.shape, Q.dtype, cache.device
    c = cache._struct(Q, "Q")
    Hq = shape[1]
    _need(Q, "Q", dtype, (cache.B, Hq, 1, cache.d), dev)
    _need(lens, "lens", torch.int32, (cache.B,), dev)
    if score and cache.score is None:
        raise ValueError("score=True needs a cache with score")
    if _elsewhere(stream, dev):
        with _on(stream, dev):
            return sage_attn_decode(Q, cache, lens, score=score, out=out, lse=lse, workspace=workspace)
    nbytes = cache._bytes.get((Hq, score))
    if nbytes is None:
        nbytes = cache._bytes[Hq, score] = lib().sage_decode_workspace_bytes(c, Hq, int(score))
    if out is not None:
        _need(out, "out", dtype, shape, dev)
    if lse is not None:
        _need(lse, "lse", torch.float32, (cache.B, Hq, 1), dev)
    _workspace_ok(workspace, dev)
    O = torch.empty_like(Q) if out is None else out
    L = torch.empty((cache.B, Hq, 1), dtype=torch.float32, device=dev) if lse is None else lse
    ws = _workspace(nbytes, dev) if workspace is None else workspace
    st = lib().sage_attn_decode(c, Hq, Q.data_ptr(), lens.data_ptr(), O.data_ptr(), L.data_ptr(), int(score), _ptr(ws),
                                nbytes if workspace is None else ws.numel() * ws.element_size(), _current(dev))
    _check("sage_attn_decode", st)
    return O, L


def sage_attn_extend(Q: torch.Tensor, cache: KvCache, start: torch.Tensor, *, count=None, out=None, lse=None,
                     workspace=None, stream=None):
    """Attention of T new tokens a sequence, Q (B,Hq,T,d), whose K and V sage_kv_append has written to slots
    start[b] + t: token t sees the slots up to its own.  count[b] of them are there (None: all T); the
    others' O is 0 and L -inf.  Hq is a multiple of the cache's heads, the cache of any kind.  A ``workspace``
    of the caller's begins at a multiple of 256 bytes.  Returns (O (B,Hq,T,d) in Q's type, L (B,Hq,T) float32)."""
    shape, dtype, dev = Q.shape, Q.dtype, cache.device
    c = cache._struct(Q, "Q")
    B, Hq, T, d = shape
    _need(Q, "Q", dtype, (cache.B, Hq, T, cache.d), dev)
    _need(start, "start", torch.int32, (cache.B,), dev)
    if count is not None:
        _need(count, "count", torch.int32, (cache.B,), dev)
    if _elsewhere(stream, dev):
        with _on(stream, dev):
            return sage_attn_extend(Q, cache, start, count=count, out=out, lse=lse, workspace=workspace)
    nbytes = cache._bytes.get(("extend", Hq, T))
    if nbytes is None:
        if len(cache._bytes) >= 4096:
            cache._bytes.clear()
        nbytes = cache._bytes["extend", Hq, T] = lib().sage_extend_workspace_bytes(c, Hq, T)
    if out is not None:
        _need(out, "out", dtype, shape, dev)
    if lse is not None:
        _need(lse, "lse", torch.float32, (B, Hq, T), dev)
    _workspace_ok(workspace, dev)
    O = torch.empty_like(Q) if out is None else out
    L = torch.empty((B, Hq, T), dtype=torch.float32, device=dev) if lse is None else lse
    ws = _workspace(nbytes, dev) if workspace is None else workspace
    st = lib().sage_attn_extend(c, Hq, T, Q.data_ptr(), start.data_ptr(), _ptr(count), O.data_ptr(), L.data_ptr(), _ptr(ws),
                                nbytes if workspace is None else ws.numel() * ws.element_size(), _current(dev))
    _check("sage_attn_extend", st)
    return O, L


def sage_kv_evict(cache: KvCache, lens: torch.Tensor, seen: torch.Tensor, *, budget: int, recent: int = 0, out=None,
                  workspace=None, stream=None) -> torch.Tensor:
    """Cuts every sequence of more than ``budget`` slots to the ``budget`` slots of the largest
    accumulated weight (cache.score), those at positions >= seen[b] - recent first; each head for
    itself, rows moved into the freed slots, ties to the lower slot (right after a prompt, whose scores
    are 0 unless the caller wrote them, its later part goes).  Returns the new lengths (B) int32, in
    ``out`` if given, which may not overlap ``lens`` or ``seen``."""
    dev = cache.device
    if cache.score is None or cache.pos is None:
        raise ValueError("eviction needs a cache with score and pos")      # (which one with scales of blocks cannot have)
    if not 0 <= recent <= budget or budget < 1:
        raise ValueError(f"budget {budget}, recent {recent}: 0 <= recent <= budget and budget >= 1 are wanted")
    budget = min(budget, cache.capacity)     # no length exceeds it
    recent = min(recent, budget)
    _need(lens, "lens", torch.int32, (cache.B,), dev)
    _need(seen, "seen", torch.int32, (cache.B,), dev)
    c = next(iter(cache._c.values()))
    nbytes = cache._bytes.get(budget)
    if nbytes is None:
        nbytes = cache._bytes[budget] = lib().sage_evict_workspace_bytes(c, budget)
    if _elsewhere(stream, dev):
        with _on(stream, dev):
            return sage_kv_evict(cache, lens, seen, budget=budget, recent=recent, out=out, workspace=workspace)
    if out is not None:
        _need(out, "out", torch.int32, (cache.B,), dev)
    _workspace_ok(workspace, dev)
    new = torch.empty_like(lens) if out is None else out
    ws = _workspace(nbytes, dev) if workspace is None else workspace
    st = lib().sage_kv_evict(c, lens.data_ptr(), seen.data_ptr(), budget, recent, new.data_ptr(), ws.data_ptr(),
                             nbytes if workspace is None else ws.numel() * ws.element_size(), _current(dev))
    _check("sage_kv_evict", st)
    return new


# ---- pages of a pool that sequences share ---------------------------------------------------


def _pages_call(name: str, cache: KvCache, ins, size: int, out, workspace, stream) -> torch.Tensor:
    """sage_kv_resize, sage_kv_fork or sage_kv_compact: int32 inputs by name, an int32 output of ``size``."""
    dev = cache.device
    if cache._pages is None:
        raise ValueError(f"{name} needs a cache with refs and held (make_kv_cache(..., pages=))")
    shape = cache.held.shape
    for what, t in ins:
        _need(t, what, torch.int32, shape, dev)
    if _elsewhere(stream, dev):
        with _on(stream, dev):
            return _pages_call(name, cache, ins, size, out, workspace, None)
    if out is None:
        out = torch.empty(size, dtype=torch.int32, device=dev)
    else:
        _need(out, "out", torch.int32, (size,), dev)
    refs, held, ws = cache._pages
    current = _current(dev)
    if workspace is not None:
        _workspace_ok(workspace, dev)
        ws = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    elif torch._C._cuda_isCurrentStreamCapturing():
        workspace = _workspace(ws[1], dev)      # the graph's: a replay finds it when the cache is gone
        ws = workspace.data_ptr(), ws[1]
    elif current not in cache._pages_streams:
        cache._pages_ws.record_stream(torch.cuda.current_stream(dev))      # not given away while this call is pending
        cache._pages_streams.add(current)
    st = getattr(lib(), name)(cache._any, refs, held, *[t.data_ptr() for _, t in ins], out.data_ptr(), *ws, current)
    _check(name, st)
    return out


def sage_kv_resize(cache: KvCache, want: torch.Tensor, *, out=None, workspace=None, stream=None) -> torch.Tensor:
    """Gives each sequence pages for ``want`` (B) int32 slots, or takes back those behind them (0: the sequence
    ends); pages are free again when no row names them.  Returns the slots that each now holds (B) int32, fewer than
    wanted where the pool has no free page left (sage_device_status() then says SAGE_ERR_PAGES)."""
    return _pages_call("sage_kv_resize", cache, (("want", want),), cache.B, out, workspace, stream)


def sage_kv_fork(cache: KvCache, parent: torch.Tensor, lens: torch.Tensor, *, out=None, workspace=None, stream=None) -> torch.Tensor:
    """Sequence b goes on as a copy of sequence ``parent[b]``, as all were before, of lens[parent[b]] slots (-1: it
    ends).  Full pages are shared, the rows of the page in use copied to a page of its own; pages of no
    sequence are free again.  Returns the new lengths (B) int32.  Sequences that then grow need
    sage_kv_resize first; one that is cut back into a page that others share must not be appended to.  Not for
    caches with score or pos."""
    if cache.score is not None or cache.pos is not None:
        raise ValueError("sage_kv_fork: a cache with score or pos is evicted from, its pages cannot be shared")
    return _pages_call("sage_kv_fork", cache, (("parent", parent), ("lens", lens)), cache.B, out, workspace, stream)


def sage_kv_compact(cache: KvCache, *, out=None, workspace=None, stream=None) -> torch.Tensor:
    """Moves the pages in use to the pool's front and lets all rows follow.  Returns their number (1) int32: the
    pool is free from there on."""
    return _pages_call("sage_kv_compact", cache, (), 1, out, workspace, stream)
