"""Thin ctypes binding of the position and cache calls of libsage_gb300.so (include/sage.h):
rotary positions, the paged key-value cache, attention of one new token over it, eviction.

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


def _kv_sizes(B: int, H: int, d: int, page: int, pages: int, max_pages: int):
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


class KvCache:
    """A paged key-value cache over tensors of the caller (struct sage_kv).

    K, V (pages,H,page,d): fp16 or bf16 values, or int8 / float8_e4m3fn codes with sK, sV
    (pages,H,page) float32, one scale a row; page a multiple of 16, B * H at most 65535.  table (B,max_pages) int32: the pages of each
    sequence; entries behind its last page are not read.  score (B,H,max_pages*page) float32 and
    pos (same, int32) are there for sage_attn_decode(score=True) and sage_kv_evict.  The tensors
    are fixed for the life of the object; their contents are the caller's and the calls'."""

    def __init__(self, K: torch.Tensor, V: torch.Tensor, table: torch.Tensor, *, sK=None, sV=None, score=None, pos=None):
        if K.dtype not in _KINDS or K.dim() != 4 or table.dim() != 2:
            raise ValueError("K must be (pages,H,page,d) in fp16, bf16, int8 or float8_e4m3fn, table (B,max_pages)")
        pages, H, page, d = K.shape
        B, max_pages = table.shape
        dev = K.device
        _kv_sizes(B, H, d, page, pages, max_pages)
        _cuda(dev)
        _need(K, "K", K.dtype, K.shape, dev)
        _need(V, "V", K.dtype, K.shape, dev)
        _need(table, "table", torch.int32, table.shape, dev)
        self.kind = _KINDS[K.dtype]
        if (self.kind == SAGE_KV_16) != (sK is None) or (sK is None) != (sV is None):
            raise ValueError("sK and sV belong to int8 and float8_e4m3fn pools, and only to them")
        for name, t in (("sK", sK), ("sV", sV)):
            if t is not None:
                _need(t, name, torch.float32, (pages, H, page), dev)
        self.capacity = max_pages * page
        for name, t, dt in (("score", score, torch.float32), ("pos", pos, torch.int32)):
            if t is not None:
                _need(t, name, dt, (B, H, self.capacity), dev)
        self.K, self.V, self.sK, self.sV, self.table, self.score, self.pos = K, V, sK, sV, table, score, pos
        self.B, self.H, self.d, self.page, self.pages, self.device = B, H, d, page, pages, dev
        # a struct for each 16-bit type that calls may bring
        types = (K.dtype,) if self.kind == SAGE_KV_16 else (torch.float16, torch.bfloat16)
        self._c = {t: ctypes.byref(SageKv(B, H, d, _DTYPES[t], self.kind, page, pages, max_pages, K.data_ptr(), V.data_ptr(),
                                          _ptr(sK), _ptr(sV), table.data_ptr(), _ptr(score), _ptr(pos))) for t in types}
        self._bytes = {}        # workspace sizes by what they depend on

    def _struct(self, t: torch.Tensor, what: str):
        """The struct for a call on 16-bit tensors like ``t``."""
        c = self._c.get(t.dtype)
        if c is None:
            raise TypeError(f"{what}: the cache takes {', '.join(map(str, self._c))}, got {t.dtype}")
        return c


def make_kv_cache(B: int, H: int, d: int, capacity: int, *, dtype=torch.int8, page: int = 64, score: bool = False,
                  device="cuda") -> KvCache:
    """A cache for B sequences of up to ``capacity`` tokens, each with pages of its own; ``score``
    adds what eviction needs.  dtype: fp16, bf16, int8 or float8_e4m3fn."""
    device = torch.device(device)
    if device.type == "cuda" and device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    m = max(1, -(-capacity // max(page, 1)))
    _kv_sizes(B, H, d, page, B * m, m)
    table = torch.arange(B * m, dtype=torch.int32, device=device).view(B, m)
    shape = (B * m, H, page, d)
    K, V = (torch.zeros(shape, dtype=dtype, device=device) for _ in range(2))
    eight = dtype in (torch.int8, torch.float8_e4m3fn)
    sK, sV = (torch.zeros(shape[:3], device=device) if eight else None for _ in range(2))
    extra = [torch.zeros((B, H, m * page), dtype=t, device=device) if score else None for t in (torch.float32, torch.int32)]
    return KvCache(K, V, table, sK=sK, sV=sV, score=extra[0], pos=extra[1])


def sage_kv_append(cache: KvCache, K: torch.Tensor, V: torch.Tensor, start: torch.Tensor, *, count=None, mu=None,
                   pos=None, stream=None) -> None:
    """Writes tokens 0 .. count[b] - 1 (None: all T) of K, V (B,H,T,d) to slots start[b] + t of the
    cache, in its form.  ``mu`` (B,H,d) float32 (8-bit caches): K-smoothing, codes of K - mu.
    ``pos`` (B) int32: position in the text of each sequence's first new token (None: its slot).
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


def sage_kv_evict(cache: KvCache, lens: torch.Tensor, seen: torch.Tensor, *, budget: int, recent: int = 0, out=None,
                  workspace=None, stream=None) -> torch.Tensor:
    """Cuts every sequence of more than ``budget`` slots to the ``budget`` slots of the largest
    accumulated weight (cache.score), those at positions >= seen[b] - recent first; each head for
    itself, rows moved into the freed slots, ties to the lower slot (right after a prompt, whose scores
    are 0 unless the caller wrote them, its later part goes).  Returns the new lengths (B) int32, in
    ``out`` if given, which may not overlap ``lens`` or ``seen``."""
    dev = cache.device
    if cache.score is None or cache.pos is None:
        raise ValueError("eviction needs a cache with score and pos")
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
