"""Python face of libiqkv's rotary positions: queries and keys normed and turned for either cache.

Argument marshalling over the C ABI only (`iq_rotary_*` in include/iqkv.h); device
memory comes from PyTorch and work is enqueued on PyTorch's current CUDA stream of
the plan's device.
"""
from __future__ import annotations

import ctypes

import numpy as np
import torch

from . import _abi
from ._abi import IQ_MAX_BATCH, IQRotaryDesc, IQRows, check, lib
from .cache import _DTYPE_CODES, _device_of, _OnDevice, _raw_stream, _stream

_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", torch.cuda.is_current_stream_capturing)
_SCALINGS = {"none": _abi.IQ_SCALING_NONE, "linear": _abi.IQ_SCALING_LINEAR, "ntk": _abi.IQ_SCALING_NTK,
             "yarn": _abi.IQ_SCALING_YARN, "banded": _abi.IQ_SCALING_BANDED}
_TURNS = {"yarn": (1.0, 32.0), "banded": (1.0, 4.0)}


def rotary_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0, original: float = 0.0,
                       low: float | None = None, high: float | None = None) -> tuple[np.ndarray, float]:
    """The radians per position of each of the rotary_dim / 2 pairs (float64) and the amplitude.

    scaling, for contexts `factor` times as long as the model's `original` length: "none"; "linear" (every frequency
    divided by factor); "ntk" (a base that grows with factor); "yarn" (pairs that turn over `high` times within the
    original length stay, those under `low` are divided, a ramp over the pairs between, and an amplitude); "banded"
    (the same limits, a ramp over the turns).  low, high: 1 and 32 for "yarn", 1 and 4 for "banded".
    """
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {', '.join(_SCALINGS)}")
    lo, hi = _TURNS.get(scaling, (0.0, 0.0))
    f = np.zeros(max(0, rotary_dim) // 2, dtype=np.float64)
    amplitude = ctypes.c_double()
    check(lib().iq_rotary_frequencies(rotary_dim, float(base), _SCALINGS[scaling], float(factor), float(original),
                                      float(lo if low is None else low), float(hi if high is None else high),
                                      f.ctypes.data, ctypes.byref(amplitude)), "iq_rotary_frequencies")
    return f, amplitude.value


def _rows(t: torch.Tensor, dtype, index: int, name: str):
    """t [entries, heads, n, 256] where it lies, if the kernels can read it there, else a copy: the tensor, its descriptor."""
    if not t.is_cuda or t.get_device() != index:
        raise ValueError(f"{name} must be a CUDA tensor on the plan's device")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}")
    if t.dim() != 4 or t.shape[3] != 256:
        raise ValueError(f"{name} must be [entries, heads, rows, 256]")
    e, h, r, d = t.stride()
    unit = 8 if dtype is torch.bfloat16 else 4  # elements in 16 bytes
    if d != 1 or (e | h | r) % unit or t.data_ptr() % 16:
        t = t.contiguous()
        e, h, r, _ = t.stride()
    if t.data_ptr() % 16:  # a contiguous slice that begins in between
        t = t.clone()
    return t, IQRows(t.data_ptr(), e, h, r)


def _positions(p: torch.Tensor, entries: int, n: int, index: int) -> torch.Tensor:
    if not p.is_cuda or p.get_device() != index or p.dtype is not torch.int32:
        raise ValueError("positions must be an int32 CUDA tensor on the plan's device")
    if p.shape != (entries, n):
        raise ValueError(f"positions must be [{entries}, {n}]")
    return p.contiguous()


class IQRotary:
    """The plan by which queries and keys are normed and turned (rotary positions), for one device.

    rotary_dim: how many leading dims turn (a multiple of 16 up to 256; 0: none).  interleaved: pairs are dims
    (2i, 2i+1), else (i, i + rotary_dim/2).  base, scaling, factor, original, low, high: see `rotary_frequencies`;
    `frequencies` (radians per position, one for each pair) takes their place, `amplitude` overrides theirs.
    q_norm, k_norm: [256] weights of the root-mean-square norm of each head's vector before it turns (None: no norm);
    they are taken as norm_offset + weight, in float32, as they are now.  Once made, a plan may be used on any stream of its
    device, and must outlive the work that uses it.
    """

    def __init__(self, rotary_dim: int = 256, base: float = 10000.0, interleaved: bool = False, scaling: str = "none", factor: float = 1.0,
                 original: float = 0.0, low: float | None = None, high: float | None = None, frequencies=None, amplitude: float | None = None,
                 q_norm: torch.Tensor | None = None, k_norm: torch.Tensor | None = None, eps: float = 1e-6, norm_offset: float = 0.0,
                 head_dim: int = 256, device=None):
        if head_dim != 256:
            raise ValueError("only head_dim 256 is built")
        if not 0 <= rotary_dim <= 256 or rotary_dim % 16:
            raise ValueError("rotary_dim must be a multiple of 16 in [0, 256]")
        if frequencies is not None:
            f, own = np.ascontiguousarray(frequencies, dtype=np.float64), 1.0
            if f.shape != (rotary_dim // 2,) or not np.isfinite(f).all():
                raise ValueError(f"frequencies must be {rotary_dim // 2} finite numbers")
        else:
            f, own = rotary_frequencies(rotary_dim, base, scaling, factor, original, low, high) if rotary_dim else (np.zeros(0), 1.0)
        self.frequencies, self.amplitude = f, float(own if amplitude is None else amplitude)
        if not np.isfinite(self.amplitude) or abs(self.amplitude) > 3e38:
            raise ValueError("amplitude must be finite")
        if (q_norm is not None or k_norm is not None) and not 1e-30 <= eps <= 3e38:
            raise ValueError("eps must be 1e-30 or more, and finite")
        for w in (q_norm, k_norm):
            if w is not None and (w.shape != (256,) or not w.is_floating_point()):
                raise ValueError("q_norm and k_norm must be 256 floating-point weights")
        if device is not None and not isinstance(device, int) and torch.device(device).type != "cuda":
            raise ValueError("device must be a CUDA device")
        self.device = _device_of(device)
        self._index, self._lib = self.device.index, lib()
        self.q_norm, self.k_norm = (None if w is None else (norm_offset + w.detach().to(self.device, torch.float32)).contiguous() for w in (q_norm, k_norm))
        self.turns = None
        if rotary_dim:
            self.turns = torch.empty(rotary_dim // 2, dtype=torch.int64, device=self.device)
            with _OnDevice(self._index):
                check(self._lib.iq_rotary_turns(f.ctypes.data, rotary_dim // 2, self.turns.data_ptr(), _stream(self._index)), "iq_rotary_turns")
        with _OnDevice(self._index):
            if not _capturing():  # (a captured plan is made when the graph is replayed)
                torch.cuda.current_stream(self.device).synchronize()
        at = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        self._desc = IQRotaryDesc(rotary_dim, 1 if interleaved else 0, self.amplitude, eps, at(self.turns), at(self.q_norm), at(self.k_norm))
        self._d = ctypes.byref(self._desc)

    def apply(self, q: torch.Tensor, k: torch.Tensor | None = None, positions=0):
        """q [entries, Hq, n, 256] and k [entries, Hkv, n, 256] normed and turned, in one launch: new
        contiguous tensors (q alone where k is None).

        bf16 or float32, views with any strides (a slice of a projection's output needs no copy where its
        rows lie at multiples of 16 bytes).  positions: of the entries' first rows, the others follow (one whole number, or
        one for each entry), or an int32 CUDA tensor [entries, n] of every row's own.  An infinity makes the
        elements that it turns into infinite or NaN; with a norm NaN, and the row's others 0.
        """
        dtype = q.dtype
        code = _DTYPE_CODES.get(dtype)
        if code is None:
            raise ValueError("q must be torch.bfloat16 or torch.float32")
        q, q_rows = _rows(q, dtype, self._index, "q")
        E, Hq, n, D = q.shape
        k_rows, Hk, k_out = None, 0, None
        if k is not None:
            k, k_rows = _rows(k, dtype, self._index, "k")
            if k.shape[0] != E or k.shape[2] != n:
                raise ValueError("q and k must have the same entries and rows")
            Hk = k.shape[1]
            k_out = torch.empty((E, Hk, n, D), dtype=dtype, device=self.device)
        if E > IQ_MAX_BATCH:
            raise ValueError(f"at most {IQ_MAX_BATCH} entries")
        start, starts, at = None, 0, None
        if type(positions) is int and -1 << 31 <= positions < 1 << 31:
            start, starts = ctypes.byref(ctypes.c_int32(positions)), 1
        elif isinstance(positions, torch.Tensor):
            positions = _positions(positions, E, n, self._index)
            at = positions.data_ptr()
        else:
            start = np.asarray(positions)
            if start.dtype.kind not in "iu" or start.ndim > 1 or (start.ndim == 1 and start.shape[0] != E):
                raise ValueError("positions must be one whole number, one for each entry, or an int32 CUDA tensor")
            if start.size and (start.min() < -1 << 31 or start.max() >= 1 << 31):
                raise ValueError("positions must fit in 32 bits")
            each = np.ascontiguousarray(start.reshape(-1), dtype=np.int32)
            start, starts = each.ctypes.data, each.shape[0]
        q_out = torch.empty((E, Hq, n, D), dtype=dtype, device=self.device)
        args = (self._d, code, ctypes.byref(q_rows), Hq, None if k is None else ctypes.byref(k_rows), Hk, E, n,
                start, starts, at, q_out.data_ptr(), None if k is None else k_out.data_ptr())
        if _device() == self._index:
            st = self._lib.iq_rotary_apply(*args, self._queue())
        else:
            with _OnDevice(self._index):
                st = self._lib.iq_rotary_apply(*args, self._queue())
        if st:
            check(st, "iq_rotary_apply")
        return q_out if k is None else (q_out, k_out)

    def _queue(self):
        """The current stream of the plan's device."""
        return _raw_stream(self._index) if _raw_stream is not None else _stream(self._index)
