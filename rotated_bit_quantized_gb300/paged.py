"""Python face of the paged 8-bit cache of libiqkv.

Argument marshalling over the C ABI only (`iq_paged_*` in include/iqkv.h);
device memory comes from PyTorch and work is enqueued on PyTorch's current
CUDA stream of the cache's device.
"""
from __future__ import annotations

import ctypes
import math
import threading

import numpy as np
import torch

from . import _abi
from ._abi import IQ_PAGE, IQPagedDesc, check, lib
from .cache import _OnDevice, _device_of, _raw_stream, _stream
from .rotary import IQRotary, _positions, _rows


_INT32 = np.dtype(np.int32)


def _ints(x, n: int | None, name: str):
    """A contiguous int32 array of `n` whole numbers (any number of them where n is None)."""
    if type(x) is np.ndarray:
        a = x
        if a.dtype is _INT32 and a.ndim == 1 and a.flags.c_contiguous and (n is None or a.shape[0] == n):
            return a
    elif type(x) is range:
        a = np.arange(x.start, x.stop, x.step)
    else:
        a = np.asarray(x if isinstance(x, (list, int, np.integer)) else list(x))
    if a.dtype is not _INT32:
        if a.size and a.dtype.kind not in "iu":
            raise ValueError(f"{name} must be whole numbers")
        wide, a = a, a.astype(_INT32)
        # (there and back as bytes takes 3 us less than comparing arrays; an unsigned one would come back from a negative)
        if a.astype(wide.dtype).tobytes() != wide.tobytes() if wide.dtype.kind == "i" else (a != wide).any():
            raise ValueError(f"{name} must fit in 32 bits")
    if n is not None and a.ndim == 0:
        a = np.full(n, a)
    if a.ndim != 1 or (n is not None and a.shape[0] != n):
        raise ValueError(f"{name} must be one whole number or {'a list of them' if n is None else n}")
    return np.ascontiguousarray(a)


def _span(window, sinks):
    """Window and sinks as the library takes them: whole numbers of 32 bits (ctypes would cut longer ones)."""
    if not (-1 << 31 <= window < 1 << 31 and -1 << 31 <= sinks < 1 << 31):
        raise ValueError("window and sinks must fit in 32 bits")
    return window, sinks


def _at(a):
    return None if a is None else a.__array_interface__["data"][0]


_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", torch.cuda.is_current_stream_capturing)


class IQPagedCache:
    """A pool of pages of 64 tokens that holds keys and values in 8 bits.

    Codes are e4m3 with one power-of-two scale per (page, kv head), keys and
    values apart; each of `slots` sequences has a row of page ids.  Pages are
    counted: `fork` lets slots share them, and an append into a page that
    others hold copies it first.  `pages` is the pool's size; `max_tokens`
    bounds one slot's length (default: the whole pool).  Keys, values and
    queries are bfloat16 and not rotated: a floating code's error is relative
    to its own element, so spreading outliers over neighbouring dims gains
    nothing.

    Wherever `slots` is an argument it lists the slots of the call's entries
    (default: the first slots, one for each entry of the tensors).

    Lengths and page ids are the host's.  Calls on one cache have to be ordered
    on one stream or by events: a page that a call releases may be handed out
    by the next one.  Host threads that call one cache are taken in turn.  A call
    captured into a CUDA graph replays with the lengths that it was captured with.
    """

    PAGE = IQ_PAGE

    def __init__(self, slots: int, kv_heads: int, pages: int, max_tokens: int | None = None, head_dim: int = 256,
                 device=None):
        self.slots, self.kv_heads, self.pages, self.head_dim = slots, kv_heads, pages, head_dim
        self.max_pages = pages if max_tokens is None else max(1, -(-max_tokens // IQ_PAGE))
        sizes = (ctypes.c_size_t * 6)()
        check(lib().iq_paged_bytes(slots, kv_heads, head_dim, pages, self.max_pages, sizes), "iq_paged_bytes")
        if device is not None and not isinstance(device, int) and torch.device(device).type != "cuda":
            raise ValueError("device must be a CUDA device")
        self.device = _device_of(device)
        self._index, self._lib = self.device.index, lib()
        dev = self.device
        self.k_codes = torch.empty((pages, kv_heads, IQ_PAGE, head_dim), dtype=torch.uint8, device=dev)
        self.v_codes = torch.empty_like(self.k_codes)
        self.k_scales = torch.empty((pages, kv_heads), dtype=torch.float32, device=dev)
        self.v_scales = torch.empty_like(self.k_scales)
        self.table = torch.empty((slots, self.max_pages), dtype=torch.int32, device=dev)
        self._status = torch.zeros(sizes[5], dtype=torch.uint8, device=dev)
        bufs = (self.k_codes, self.v_codes, self.k_scales, self.v_scales, self.table, self._status)
        assert [t.numel() * t.element_size() for t in bufs] == list(sizes)
        self._lens = np.zeros(slots, dtype=np.int32)
        self._table = np.zeros((slots, self.max_pages), dtype=np.int32)
        self._refs = np.zeros(pages, dtype=np.int32)
        self._lock = threading.RLock()  # the library's calls run without the interpreter's
        self._need, self._scratch, self._scale = {}, {}, 1.0 / math.sqrt(head_dim)
        self._desc = IQPagedDesc()
        self._d = ctypes.byref(self._desc)
        check(lib().iq_paged_alloc(self._d, slots, kv_heads, head_dim, pages, self.max_pages,
                                   (ctypes.c_void_p * 6)(*[t.data_ptr() for t in bufs]),
                                   _at(self._lens), _at(self._table), _at(self._refs)), "iq_paged_alloc")

    def _run(self, f, *args) -> None:
        """Call a library function with the cache's device current, one thread at a time."""
        with self._lock:
            if _device() == self._index:
                code = f(*args)
            else:
                with _OnDevice(self._index):
                    code = f(*args)
            if code:
                check(code, f.__name__)

    def _queue(self):
        """The current stream of the cache's device."""
        return _raw_stream(self._index) if _raw_stream is not None else _stream(self._index)

    # ---------------------------------------------------------------- state
    @property
    def lens(self) -> np.ndarray:
        """The slots' lengths, int32 [slots] (a copy)."""
        with self._lock:
            return self._lens.copy()

    @property
    def pages_free(self) -> int:
        return self._desc.free_pages

    @property
    def pages_used(self) -> int:
        return self.pages - self._desc.free_pages

    @property
    def nbytes(self) -> int:
        """Bytes of the pool and the table."""
        return sum(t.numel() * t.element_size()
                   for t in (self.k_codes, self.v_codes, self.k_scales, self.v_scales, self.table))

    def page_ids(self, slot: int) -> np.ndarray:
        """The page ids of a slot, in order (a copy)."""
        with self._lock:
            return self._table[slot, : -(-int(self._lens[slot]) // IQ_PAGE)].copy()

    def device_status(self) -> int:
        """Synchronise, return the kernels' status word (0: all normal) and clear it."""
        st = ctypes.c_int()
        with _OnDevice(self._index):
            code = lib().iq_read_status(self._status.data_ptr(), _stream(self._index), ctypes.byref(st))
        if code not in (_abi.IQ_OK, _abi.IQ_ERR_DEVICE):
            check(code, "iq_read_status")
        return st.value

    # ---------------------------------------------------------------- arguments
    def _tensor(self, t: torch.Tensor, name: str) -> torch.Tensor:
        if not t.is_cuda or t.get_device() != self._index:
            raise ValueError(f"{name} must be a CUDA tensor on {self.device}")
        if t.dtype is not torch.bfloat16:
            raise ValueError(f"{name} must be torch.bfloat16")
        if t.dim() != 4 or t.shape[3] != self.head_dim:
            raise ValueError(f"{name} must be [entries, heads, rows, {self.head_dim}]")
        return t.contiguous()

    def _rows(self, keys, values):
        keys, values = self._tensor(keys, "keys"), self._tensor(values, "values")
        if keys.shape != values.shape or keys.shape[1] != self.kv_heads:
            raise ValueError("keys/values must be [entries, Hkv, n, D]")
        return keys, values

    def _entries(self, n: int, slots, counts):
        """slots, counts as int32 arrays of n entries, or None for the defaults."""
        if slots is None and n > self.slots:
            raise ValueError(f"{n} entries for {self.slots} slots")
        return (None if slots is None else _ints(slots, n, "slots"),
                None if counts is None else _ints(counts, n, "counts"))

    def _outputs(self, q, counts, out, out_dtype):
        if out is None:  # rows that do not exist are left as they are: zeros
            if out_dtype is None and counts is None:
                return torch.empty_like(q)
            dtype = out_dtype or torch.bfloat16
            if dtype not in (torch.float32, torch.bfloat16):
                raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
            return torch.empty_like(q, dtype=dtype) if counts is None else torch.zeros_like(q, dtype=dtype)
        if out.dtype not in (torch.float32, torch.bfloat16) or not out.is_contiguous():
            raise ValueError("out must be a contiguous bf16 or f32 tensor")
        if out.shape != q.shape or out.device != q.device or (out_dtype or out.dtype) != out.dtype:
            raise ValueError("out must have q's shape and device, and out_dtype")
        at, to = q.data_ptr(), out.data_ptr()
        if to < at + q.numel() * 2 and at < to + out.numel() * out.element_size():
            raise ValueError("out must not overlap q")
        return out

    def _workspace(self, q_heads: int, rows: int, entries: int, stream, shared: bool):
        """Scratch for a call on `stream`: one per stream, kept, as work on one stream is in order
        (so the lock is held from here until the call has made its launches); for a captured
        call its own, as graphs captured on one stream may run at once."""
        key = (q_heads, rows, entries, shared)
        need = self._need.get(key)
        if need is None:
            c = ctypes.c_size_t()
            self._run(self._lib.iq_paged_attend_shared_workspace if shared else self._lib.iq_paged_attend_workspace, self._d, q_heads, rows, entries, ctypes.byref(c))
            if len(self._need) > 256:
                self._need.clear()
            need = self._need[key] = c.value
        if _device() == self._index:
            captured = _capturing()
        else:
            with _OnDevice(self._index):
                captured = _capturing()
        if captured:
            return torch.empty(need, dtype=torch.uint8, device=self.device)
        ws = self._scratch.get(stream)
        if ws is None or ws.numel() < need:
            if len(self._scratch) > 16:
                self._scratch.clear()
            ws = self._scratch[stream] = torch.empty(max(need, 1 << 20), dtype=torch.uint8, device=self.device)
        return ws

    # ---------------------------------------------------------------- rows
    def append(self, keys: torch.Tensor, values: torch.Tensor, slots=None, counts=None) -> None:
        """Quantise and append rows: entry i's first counts[i] rows (default: all n) to slots[i].

        keys, values: bf16 CUDA tensors [entries, Hkv, n, D].  Raises IQError
        (capacity) when the pool or a slot is too small; nothing has changed then.
        """
        keys, values = self._rows(keys, values)
        E, _, n, _ = keys.shape
        slots, counts = self._entries(E, slots, counts)
        self._run(self._lib.iq_paged_append, self._d, keys.data_ptr(), values.data_ptr(), n, _at(slots), _at(counts), E, self._queue())

    def append_rotary(self, q: torch.Tensor | None, keys: torch.Tensor, values: torch.Tensor, rotary: IQRotary, slots=None, counts=None,
                      positions: torch.Tensor | None = None) -> torch.Tensor | None:
        """`append` of a projection's rows as they are, in one launch: queries and keys normed and turned by `rotary`
        at the positions where the rows come to stand (or at positions, an int32 CUDA tensor [entries, n]), keys and values quantised into
        the pages.  Returns the queries for `attend`, [entries, Hq, n, D] (None where q is None).

        q [entries, Hq, n, D], keys, values [entries, Hkv, n, D]: bf16 CUDA tensors, views with any strides (see
        `IQRotary.apply`).  Rows behind counts[i] are not read; their queries come back as zeros.  Keys
        are held as the codes nearest to what the formula gives without any rounding, from the plan's
        weights (norm_offset + weight in float32), frequencies and amplitude.
        """
        if rotary._index != self._index:
            raise ValueError("the rotary plan must be on the cache's device")
        keys, k_rows = _rows(keys, torch.bfloat16, self._index, "keys")
        values, v_rows = _rows(values, torch.bfloat16, self._index, "values")
        if keys.shape != values.shape or keys.shape[1] != self.kv_heads:
            raise ValueError("keys/values must be [entries, Hkv, n, D]")
        E, _, n, D = keys.shape
        q_rows, Hq, out = None, 0, None
        if q is not None:
            q, q_rows = _rows(q, torch.bfloat16, self._index, "q")
            if q.shape[0] != E or q.shape[2] != n:
                raise ValueError("keys/values and q must have the same entries and rows")
            Hq = q.shape[1]
        slots, counts = self._entries(E, slots, counts)
        at = None
        if positions is not None:
            positions = _positions(positions, E, n, self._index)
            at = positions.data_ptr()
        if q is not None:
            out = torch.empty((E, Hq, n, D), dtype=torch.bfloat16, device=self.device)
        self._run(self._lib.iq_paged_append_rotary, self._d, rotary._d, None if q is None else ctypes.byref(q_rows), Hq, ctypes.byref(k_rows),
                  ctypes.byref(v_rows), n, _at(slots), _at(counts), E, at, None if q is None else out.data_ptr(), self._queue())
        return out

    def read(self, start, n: int, slots=None) -> tuple[torch.Tensor, torch.Tensor]:
        """The values held in rows [start, start + n) of the slots (default: all), as bf16
        (exact): keys, values [entries, Hkv, n, D]; rows past a slot's length are 0.
        start: one position, or one for each entry."""
        entries = self.slots if slots is None else len(slots)
        slots, _ = self._entries(entries, slots, None)
        start = _ints(start, entries, "start")
        if n < 0:
            raise ValueError("n must not be negative")
        keys = torch.empty((entries, self.kv_heads, n, self.head_dim), dtype=torch.bfloat16, device=self.device)
        values = torch.empty_like(keys)
        self._run(self._lib.iq_paged_read, self._d, _at(slots), _at(start), entries, n, keys.data_ptr(), values.data_ptr(), self._queue())
        return keys, values

    def trim(self, n, slots=None) -> np.ndarray:
        """Drop up to n tokens (one number, or one for each entry) from the end of the slots and
        release the pages left empty; returns the counts dropped."""
        entries = self.slots if slots is None else len(slots)
        slots, _ = self._entries(entries, slots, None)
        n = _ints(n, entries, "n")
        out = np.zeros(entries, dtype=np.int32)
        self._run(self._lib.iq_paged_trim, self._d, _at(slots), _at(n), entries, _at(out))
        return out

    # ---------------------------------------------------------------- pages
    def free(self, slots) -> None:
        """Release every page of these slots."""
        slots = _ints(slots, None, "slots")
        self._run(self._lib.iq_paged_free, self._d, _at(slots), len(slots))

    def fork(self, src, dst) -> None:
        """Make each slot dst[i] a second holder of slot src[i]'s pages; what dst[i] held is released.
        No codes are copied.  All at once: a source is what it was before the call."""
        dst = _ints(dst, None, "dst")
        src = _ints(src, len(dst), "src")
        self._run(self._lib.iq_paged_fork, self._d, _at(src), _at(dst), len(dst), self._queue())

    def compact(self, out: "IQPagedCache | None" = None) -> "IQPagedCache":
        """A copy of this cache that holds each live page once, lowest ids first; sharing is kept.
        `out`: the cache to fill (what it held is dropped); by default a new one with a pool
        of just the live pages.  Grows or shrinks a pool, takes and restores snapshots."""
        if out is None:
            out = IQPagedCache(self.slots, self.kv_heads, max(1, self.pages_used), self.max_pages * IQ_PAGE,
                               self.head_dim, self.device)
        elif out.device != self.device:
            raise ValueError("out must be on the cache's device")
        first, second = sorted((self, out), key=id)  # the same order in every thread
        with first._lock, second._lock:
            self._run(self._lib.iq_paged_compact, self._d, out._d, self._queue())
        return out

    # ---------------------------------------------------------------- attention
    def attend(self, q: torch.Tensor, causal: bool = True, scale: float | None = None, window: int = 0,
               sinks: int = 0, slots=None, counts=None, out: torch.Tensor | None = None, out_dtype=None,
               shared: bool = False) -> torch.Tensor:
        """Attention of q [entries, Hq, L, D] (bf16) over the slots' pages; returns [entries, Hq, L, D].

        The L queries stand at each slot's last L positions (its last counts[i],
        where counts are given: the queries behind them do not exist, and their
        rows of `out` are left as they were).  `out` must not overlap q.  causal: a query sees the keys
        up to its own position; `window` > 0: only the last `window` of them, and
        the slot's first `sinks` tokens.  A query that sees nothing gets 0.
        Softmax weights are held to 2^-8 of each, sums in float32, whatever out_dtype is.
        shared: read pages that several of the slots hold (forked paths, a common prompt) once for all of
        them, where an estimate says that this is faster (of 20000 random calls 0.4% took 8% longer, or more, the worst 1.4 times as long); a
        call captured so replays with the sharing it was captured with.
        """
        q = self._tensor(q, "q")
        E, Hq, L, D = q.shape
        slots, counts = self._entries(E, slots, counts)
        out = self._outputs(q, counts, out, out_dtype)
        window, sinks = _span(window, sinks)
        stream = self._queue()
        with self._lock:
            ws = self._workspace(Hq, L, E, stream, shared)
            self._run(self._lib.iq_paged_attend_shared if shared else self._lib.iq_paged_attend, self._d, q.data_ptr(), Hq, L, _at(slots), _at(counts), E,
                      self._scale if scale is None else scale, 1 if causal else 0, window, sinks, out.data_ptr(),
                      1 if out.dtype is torch.float32 else 0, ws.data_ptr(), ws.numel(), stream)
        return out

    def append_attend(self, keys: torch.Tensor, values: torch.Tensor, q: torch.Tensor, causal: bool = True,
                      scale: float | None = None, window: int = 0, sinks: int = 0, slots=None, counts=None,
                      out: torch.Tensor | None = None, out_dtype=None, shared: bool = False) -> torch.Tensor:
        """`append(keys, values)` then `attend(q)` of the same entries in one library call: the step of
        a decode loop or one chunk of a prompt."""
        keys, values = self._rows(keys, values)
        q = self._tensor(q, "q")
        E, Hq, L, D = q.shape
        if keys.shape[0] != E:
            raise ValueError("keys/values and q must have the same entries")
        slots, counts = self._entries(E, slots, counts)
        out = self._outputs(q, counts, out, out_dtype)
        window, sinks = _span(window, sinks)
        stream = self._queue()
        with self._lock:
            ws = self._workspace(Hq, L, E, stream, shared)
            self._run(self._lib.iq_paged_append_attend_shared if shared else self._lib.iq_paged_append_attend, self._d, keys.data_ptr(), values.data_ptr(), keys.shape[2], q.data_ptr(), Hq, L,
                      _at(slots), _at(counts), E, self._scale if scale is None else scale, 1 if causal else 0, window, sinks,
                      out.data_ptr(), 1 if out.dtype is torch.float32 else 0, ws.data_ptr(), ws.numel(), stream)
        return out
