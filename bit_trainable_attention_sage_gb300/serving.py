"""Thin ctypes binding of the position and cache calls of libsage_gb300.so (include/sage.h).

As in binding.py, every function has the name of the C entry point it wraps, checks and marshals
its arguments, and takes outputs and workspaces from PyTorch; nothing is computed here.  Calls run
on ``stream`` or else on the current stream of the tensors' device; what a call allocates belongs
to that stream.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from .binding import SAGE_BF16, SAGE_FP16, _check, lib

SAGE_FP32 = 2
_DTYPES = {torch.float16: SAGE_FP16, torch.bfloat16: SAGE_BF16, torch.float32: SAGE_FP32}


class SageRopeParams(ctypes.Structure):
    """struct sage_rope_params (include/sage.h)."""
    _fields_ = [(n, ctypes.c_int) for n in ("B", "H", "Hk", "N", "d", "dtype", "axes", "pos_batch", "rotary",
                                            "interleaved", "inverse")] + \
               [("sections", ctypes.POINTER(ctypes.c_int)), ("freq", ctypes.POINTER(ctypes.c_double))]


def _need(t: torch.Tensor, what: str, dtype, shape, device):
    """A contiguous tensor of this type and shape on this device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what}: must be a contiguous CUDA tensor on {device}")


@contextlib.contextmanager
def _on(stream, device):
    """Makes ``stream`` (or the device's current stream) current, so that the launch and what is
    allocated for it belong to the same stream and device; yields its handle."""
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
        with torch.cuda.stream(stream):
            yield stream.cuda_stream
    elif torch.cuda.current_device() != device.index:
        with torch.cuda.device(device):
            yield torch.cuda.current_stream().cuda_stream
    else:
        yield torch.cuda.current_stream().cuda_stream


# ---- rotary positions -----------------------------------------------------------------------


class Rope:
    """What a rotation is besides its positions: made once by make_rope."""

    def __init__(self, d: int, sections, freqs, interleaved: bool):
        self.d, self.sections, self.freqs, self.interleaved = d, tuple(sections), tuple(freqs), bool(interleaved)
        self.axes, self.rotary = len(self.sections), 2 * sum(self.sections)
        self._sections = (ctypes.c_int * self.axes)(*self.sections)
        self._freq = (ctypes.c_double * len(self.freqs))(*self.freqs)


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
    B, H, N, d = Q.shape
    dev = Q.device
    if Q.dtype not in _DTYPES:
        raise TypeError(f"sage_rope takes fp16, bf16 or float32 tensors, got {Q.dtype}")
    _need(Q, "Q", Q.dtype, Q.shape, dev)
    if d != rope.d:
        raise ValueError(f"Q has {d} channels, the rope {rope.d}")
    Hk = 0
    if K is not None:
        Hk = K.shape[1]
        _need(K, "K", Q.dtype, (B, Hk, N, d), dev)
    pb = 1 if positions.dim() == 3 and positions.shape[1] == 1 else B
    _need(positions, "positions", torch.int32, (rope.axes, pb, N), dev)
    with _on(stream, dev) as st:
        if out is None:
            Qo, Ko = torch.empty_like(Q), None if K is None else torch.empty_like(K)
        else:
            Qo, Ko = out
            _need(Qo, "out[0]", Q.dtype, Q.shape, dev)
            if K is not None:
                _need(Ko, "out[1]", K.dtype, K.shape, dev)
        p = SageRopeParams(B, H, Hk, N, d, _DTYPES[Q.dtype], rope.axes, pb, rope.rotary, rope.interleaved, bool(inverse),
                           rope._sections, rope._freq)
        _check("sage_rope", lib().sage_rope(ctypes.byref(p), Q.data_ptr(), None if K is None else K.data_ptr(),
                                            positions.data_ptr(), Qo.data_ptr(), None if K is None else Ko.data_ptr(), st))
    return Qo, Ko
