"""The paged 8-bit cache's host side: sizes, refusals, page counting.  Runs
without a GPU: device pointers are made up and never followed."""
import ctypes

import numpy as np
import pytest
import torch

INVALID, CAPACITY, WORKSPACE, UNSUPPORTED, CUDA = 1, 2, 3, 4, 5
P = ctypes.c_void_p(0x20000000)


@pytest.fixture(scope="module")
def L():
    from rotated_bit_quantized_gb300 import build
    build.build()
    from rotated_bit_quantized_gb300 import _abi
    return _abi.lib()


class Fake:
    """A descriptor over host arrays of its own and made-up device addresses."""

    def __init__(self, L, slots=4, heads=2, pages=20, max_pages=8, base=0x10000000):
        from rotated_bit_quantized_gb300._abi import IQPagedDesc
        self.L, self.d = L, IQPagedDesc()
        self.lens, self.refs = np.full(slots, 7, dtype=np.int32), np.full(pages, 7, dtype=np.int32)
        self.table = np.full((slots, max_pages), 7, dtype=np.int32)
        bufs = (ctypes.c_void_p * 6)(*[base + i * 0x1000000 for i in range(6)])
        self.p = ctypes.byref(self.d)
        assert L.iq_paged_alloc(self.p, slots, heads, 256, pages, max_pages, bufs, self.lens.ctypes.data,
                                self.table.ctypes.data, self.refs.ctypes.data) == 0

    def hold(self, slot, ids, length):
        """Give a slot pages as an append would have."""
        self.table[slot, : len(ids)] = ids
        self.lens[slot] = length
        for i in ids:
            if self.refs[i] == 0:
                self.d.free_pages -= 1
            self.refs[i] += 1

    def state(self):
        return (self.lens.tolist(), self.refs.tolist(), self.d.free_pages,
                [self.table[s, : -(-int(self.lens[s]) // 64)].tolist() for s in range(len(self.lens))])

    def append(self, n, slots=None, counts=None, k=4):
        return self.L.iq_paged_append(self.p, P, P, n, ints(slots), ints(counts), k, None)

    def attend(self, Hq=4, n=1, slots=None, counts=None, k=4, scale=0.1, causal=1, window=0, sinks=0, out_f32=0, q=P,
               out=P, ws=P, nbytes=1 << 40):
        return self.L.iq_paged_attend(self.p, q, Hq, n, ints(slots), ints(counts), k, scale, causal, window, sinks, out,
                                      out_f32, ws, nbytes, None)


_keep = []


def ints(x):
    if x is None:
        return None
    a = np.array(x, dtype=np.int32)
    _keep.append(a)
    return a.ctypes.data


def test_bytes(L):
    out = (ctypes.c_size_t * 6)()
    assert L.iq_paged_bytes(3, 2, 256, 10, 5, out) == 0
    assert list(out) == [10 * 2 * 64 * 256] * 2 + [10 * 2 * 4] * 2 + [3 * 5 * 4, 8448]
    for bad in [(0, 2, 256, 10, 5), (3, 0, 256, 10, 5), (3, 2, 0, 10, 5), (3, 2, 256, 0, 5), (3, 2, 256, 10, 0), (-1, 2, 256, 10, 5)]:
        assert L.iq_paged_bytes(*bad, out) == INVALID, bad
    for bad in [(3, 2, 128, 10, 5), (257, 2, 256, 10, 5), (3, 1025, 256, 10, 5), (3, 2, 256, 1 << 24, 5), (3, 2, 256, 10, 1 << 25)]:
        assert L.iq_paged_bytes(*bad, out) == UNSUPPORTED, bad
    assert L.iq_paged_bytes(3, 2, 256, (1 << 24) - 1, 5, out) == 0 and out[0] == ((1 << 24) - 1) * 2 * 64 * 256  # past 32 bits
    assert L.iq_paged_bytes(3, 2, 256, 10, 5, None) == INVALID


def test_alloc_and_check(L):
    f = Fake(L)
    assert f.state() == ([0] * 4, [0] * 20, 20, [[]] * 4) and f.table.sum() == 0
    assert L.iq_paged_check(f.p) == 0 and L.iq_paged_check(None) == INVALID
    for field, bad in [("k_codes", 0), ("v_scales", 0x10000008), ("table", 0), ("status", 0x10000004), ("lens", 0), ("refs", 0),
                       ("table_host", 0), ("free_pages", 21), ("free_pages", -1), ("first_free", -1), ("kv_heads", 0)]:
        f = Fake(L)
        setattr(f.d, field, bad)
        assert L.iq_paged_check(f.p) == INVALID, field
    f = Fake(L)
    f.lens[2] = 8 * 64 + 1
    assert L.iq_paged_check(f.p) == INVALID
    f.lens[2] = -1
    assert L.iq_paged_check(f.p) == INVALID


def test_trim_and_free_count_pages(L):
    f = Fake(L)
    f.hold(0, [3, 0, 5], 130)
    f.hold(1, [3, 0, 6], 129)   # shares two pages with slot 0
    assert f.d.free_pages == 16
    out = np.zeros(2, dtype=np.int32)
    assert L.iq_paged_trim(f.p, ints([1, 2]), ints([1, 9]), 2, out.ctypes.data) == 0
    assert out.tolist() == [1, 0] and f.lens.tolist() == [130, 128, 0, 0] and f.refs[6] == 0 and f.d.free_pages == 17
    assert L.iq_paged_trim(f.p, ints([0]), ints([1000]), 1, None) == 0  # all of slot 0: the shared pages stay
    assert f.refs[[0, 3, 5]].tolist() == [1, 1, 0] and f.d.free_pages == 18 and f.lens[0] == 0
    assert L.iq_paged_free(f.p, ints([1, 0]), 2) == 0
    assert f.state() == ([0] * 4, [0] * 20, 20, [[]] * 4) and f.d.first_free == 0
    for slots, n, k in [([0, 0], [1, 1], 2), ([4], [1], 1), ([-1], [1], 1), ([0], [-1], 1), (None, [1] * 5, 5), ([0], None, 1)]:
        assert L.iq_paged_trim(f.p, ints(slots), ints(n), k, None) == INVALID
    assert L.iq_paged_free(f.p, ints([9]), 1) == INVALID


def test_append_refusals_change_nothing(L):
    f = Fake(L)
    f.hold(0, [0, 1], 100)
    f.hold(1, [0, 1], 100)
    was = f.state()
    assert f.append(-1) == INVALID
    assert f.append(1, slots=[0, 1, 2, 2]) == INVALID
    assert f.append(1, slots=[0, 1, 2, 4]) == INVALID
    assert f.append(1, k=5) == INVALID
    assert f.append(1, k=-1) == INVALID
    assert f.append(3, counts=[1, 2, 4, 0]) == INVALID
    assert f.append(3, counts=[1, 2, -1, 0]) == INVALID
    assert f.append(8 * 64 + 1, slots=[2], k=1) == CAPACITY               # past a slot's row
    assert f.append(8 * 64 - 99, slots=[0], k=1) == CAPACITY
    assert f.append(64 * 7, slots=[2, 3, 0], counts=[448, 448, 256], k=3) == CAPACITY  # 7 + 7 + 4 and a copy: 19 of 18
    assert L.iq_paged_append(f.p, None, P, 1, None, None, 4, None) == INVALID
    assert L.iq_paged_append(f.p, P, ctypes.c_void_p(0x20000008), 1, None, None, 4, None) == INVALID
    assert f.state() == was
    assert f.append(0) == 0 and f.append(5, counts=[0] * 4) == 0 and f.append(3, k=0) == 0  # nothing to do
    assert f.state() == was


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up device addresses: only where every launch fails")
def test_a_failed_launch_puts_everything_back(L):
    f = Fake(L)
    f.hold(0, [2, 1], 100)
    f.hold(1, [2, 1], 100)
    f.hold(2, [5], 64)
    was = f.state()
    assert f.append(200) == CUDA and f.state() == was
    assert f.append(1, slots=[1, 0], k=2) == CUDA and f.state() == was   # two copies of the shared page
    assert L.iq_paged_fork(f.p, ints([0]), ints([3]), 1, None) == CUDA and f.state() == was
    g = Fake(L, base=0x40000000)
    assert L.iq_paged_compact(f.p, g.p, None) == CUDA and g.state() == ([0] * 4, [0] * 20, 20, [[]] * 4)
    assert L.iq_paged_append_attend(f.p, P, P, 1, P, 4, 1, None, None, 4, 0.1, 1, 0, 0, P, 0, P, 1 << 40, None) == CUDA
    assert f.state() == was


def test_fork_refusals_and_empty_sources(L):
    f = Fake(L)
    f.hold(0, [0], 10)
    was = f.state()
    for src, dst in [([0, 0], [1, 1]), ([4], [1]), ([0], [-1]), (None, [1]), ([0], None)]:
        assert L.iq_paged_fork(f.p, ints(src), ints(dst), len(dst or src), None) == INVALID
    assert L.iq_paged_fork(f.p, ints([0] * 300), ints([0] * 300), 300, None) == INVALID
    assert L.iq_paged_fork(f.p, None, None, 0, None) == 0 and f.state() == was
    assert L.iq_paged_fork(f.p, ints([1]), ints([0]), 1, None) == 0      # an empty source: slot 0 is released, no launch
    assert f.state() == ([0] * 4, [0] * 20, 20, [[]] * 4)


def test_compact_refusals(L):
    f = Fake(L)
    f.hold(0, [4, 9], 100)
    assert L.iq_paged_compact(f.p, f.p, None) == INVALID
    assert L.iq_paged_compact(f.p, Fake(L, slots=5, base=0x40000000).p, None) == INVALID
    assert L.iq_paged_compact(f.p, Fake(L, heads=1, base=0x40000000).p, None) == INVALID
    assert L.iq_paged_compact(f.p, Fake(L).p, None) == INVALID           # common buffers
    assert L.iq_paged_compact(f.p, Fake(L, pages=1, base=0x40000000).p, None) == CAPACITY
    assert L.iq_paged_compact(f.p, Fake(L, max_pages=1, base=0x40000000).p, None) == CAPACITY
    g = Fake(L, base=0x40000000)
    g.hold(1, [0, 1, 2], 190)
    assert L.iq_paged_compact(Fake(L).p, g.p, None) == 0                 # an empty source: dst is emptied, no launch
    assert g.state() == ([0] * 4, [0] * 20, 20, [[]] * 4)


def test_attend_refusals(L):
    f = Fake(L)
    f.hold(0, [0], 10)
    for kw in [dict(causal=2), dict(window=-1), dict(sinks=-1), dict(window=3, causal=0), dict(sinks=2), dict(out_f32=2),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(counts=[0, 0, 0, 2]), dict(counts=[-1, 0, 0, 0]),
               dict(slots=[0, 1, 2, 4]), dict(k=5), dict(k=257), dict(Hq=0), dict(n=-1), dict(q=None), dict(out=None),
               dict(q=ctypes.c_void_p(0x20000002)), dict(out=ctypes.c_void_p(0x20000008))]:
        assert f.attend(**kw) == INVALID, kw
    for kw in [dict(Hq=3), dict(Hq=2 * 65), dict(n=1 << 30)]:
        assert f.attend(**kw) == UNSUPPORTED, kw
    need = ctypes.c_size_t(0)
    assert L.iq_paged_attend_workspace(f.p, 4, 1, 4, ctypes.byref(need)) == 0
    assert L.iq_paged_attend_workspace(f.p, 4, 1, 4, None) == INVALID
    if need.value:
        assert f.attend(ws=None) == WORKSPACE
        assert f.attend(nbytes=need.value - 1) == WORKSPACE
        assert f.attend(ws=ctypes.c_void_p(0x20000010)) == WORKSPACE
    assert f.attend(n=0) == 0 and f.attend(k=0) == 0                     # nothing to do


def test_outputs_over_the_queries_are_refused():
    from rotated_bit_quantized_gb300.paged import IQPagedCache

    def given(q, out):
        return IQPagedCache._outputs(None, q, None, out, None)
    x = torch.zeros(6, 2, 3, 256, dtype=torch.bfloat16)
    wide = x.view(torch.float32).view(3, 2, 3, 256)                       # the same memory as fp32 rows
    for q, out in [(x[:2], x[2:4]), (x[2:4], x[:2]), (x[4:5], wide[:1]), (x[:1], wide[1:2])]:   # side by side, apart
        assert given(q, out) is out
    for q, out in [(x, x), (x[:2], x[1:3]), (x[1:3], x[:2]), (x[1:2], wide[:1]), (x[:1], wide[:1])]:
        with pytest.raises(ValueError, match="overlap"):
            given(q, out)


def test_append_attend_checks_both_first(L):
    f = Fake(L)
    f.hold(0, [0], 10)
    was = f.state()

    def call(n=1, nq=1, slots=None, counts=None, k=4, Hq=4, window=0):
        return L.iq_paged_append_attend(f.p, P, P, n, P, Hq, nq, ints(slots), ints(counts), k, 0.1, 1, window, 0, P, 0, P,
                                        1 << 40, None)
    assert call(Hq=3) == UNSUPPORTED
    assert call(window=-1) == INVALID
    assert call(n=2, counts=[1, 1, 1, 1]) == INVALID                     # counts with other numbers of rows and queries
    assert call(slots=[0, 1, 1, 2]) == INVALID
    assert call(n=600) == CAPACITY
    assert f.state() == was


def test_calls_with_too_many_tiles_are_refused_before_the_append(L):
    """2^29 query rows, 2^22 units of 128, over 512 tiles of keys: 2^31 tiles."""
    def call(f, nq, causal, n=64, k=1):
        return L.iq_paged_append_attend(f.p, P, P, n, P, 1, nq, None, None, k, 0.1, causal, 0, 0,
                                        ctypes.c_void_p(1 << 44), 0, ctypes.c_void_p(0x40000000), 1 << 40, None)
    f = Fake(L, slots=1, heads=1, pages=1024, max_pages=1024)
    f.hold(0, list(range(1023)), 1023 * 64)
    was = f.state()
    assert call(f, 1 << 29, 0) == UNSUPPORTED and f.state() == was
    assert f.attend(Hq=1, n=1 << 29, k=1, causal=0, out=ctypes.c_void_p(1 << 44), ws=ctypes.c_void_p(0x40000000)) == UNSUPPORTED
    if not torch.cuda.is_available():  # a bound passes 2^31, the tiles do not: causal rows before the first key see one tile each
        assert call(f, 1 << 29, 1) == CUDA and f.state() == was


def test_read_refusals(L):
    f = Fake(L)
    f.hold(0, [0], 10)

    def call(slots=None, start=(0, 0, 0, 0), k=4, n=3, ko=P, vo=P):
        return L.iq_paged_read(f.p, ints(slots), ints(start), k, n, ko, vo, None)
    assert call(start=(0, 0, 0, -1)) == INVALID
    assert call(slots=[0, 1, 2, 4]) == INVALID
    assert call(n=-1) == INVALID
    assert call(start=None) == INVALID
    assert call(ko=None) == INVALID and call(vo=ctypes.c_void_p(0x20000004)) == INVALID
    assert call(n=0) == 0 and call(k=0) == 0


def test_integer_arguments():
    from rotated_bit_quantized_gb300.paged import _ints
    assert _ints(5, 3, "x").tolist() == [5, 5, 5] and _ints(range(2), None, "x").dtype == np.int32
    assert _ints(np.array([1, 2], dtype=np.int64), 2, "x").tolist() == [1, 2]
    for bad, n in [([1, 2], 3), ([1.5], 1), ([[1]], None), ([2**31], 1), ([-2**31 - 1], 1), (3, None)]:
        with pytest.raises(ValueError):
            _ints(bad, n, "x")


def test_window_and_sinks_fit_in_32_bits():
    from rotated_bit_quantized_gb300.paged import _span
    assert _span(2**31 - 1, 2**31 - 1) == (2**31 - 1, 2**31 - 1) and _span(-1, 0) == (-1, 0)
    for bad in [(2**31, 0), (2**32 + 5, 0), (5, 2**32), (-2**31 - 1, 0)]:
        with pytest.raises(ValueError):
            _span(*bad)


def test_host_threads_take_turns(monkeypatch):
    """Library calls drop the interpreter's lock; a call and its choice of scratch must not be torn apart."""
    import threading
    import time

    from rotated_bit_quantized_gb300 import paged
    c = paged.IQPagedCache.__new__(paged.IQPagedCache)
    c.device, c._index, c.slots, c.kv_heads, c.head_dim, c._d, c._scale = torch.device("cuda", 0), 0, 4, 2, 256, None, 1 / 16
    c._lock, c._scratch, c._need = threading.RLock(), {}, {}
    c._lens = np.zeros(4, dtype=np.int32)
    inside, seen = [], []

    class Lib:
        def busy(self, *args):
            inside.append(1)
            seen.append(len(inside))
            time.sleep(0.002)
            inside.pop()
            return 0
        iq_paged_append = iq_paged_attend = iq_paged_append_attend = iq_paged_trim = iq_paged_read = busy
    c._lib = Lib()
    monkeypatch.setattr(paged, "_device", lambda: 0)
    monkeypatch.setattr(c.__class__, "_tensor", lambda self, t, name: t)
    monkeypatch.setattr(c.__class__, "_queue", lambda self: 0)
    monkeypatch.setattr(c.__class__, "_workspace", lambda self, *a: inside.append(1) or time.sleep(0.001) or inside.pop() and torch.empty(1))
    x, q = torch.zeros(4, 2, 1, 256, dtype=torch.bfloat16), torch.zeros(4, 8, 1, 256, dtype=torch.bfloat16)

    def work():
        for _ in range(5):
            c.append(x, x), c.attend(q), c.append_attend(x, x, q), c.trim(1), c.lens
    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert seen == [1] * (4 * 5 * 4)


def test_device_arguments(L, monkeypatch):
    from rotated_bit_quantized_gb300 import IQPagedCache
    from rotated_bit_quantized_gb300.cache import _device_of
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    assert _device_of(None) == _device_of("cuda") == torch.device("cuda", 1)
    assert _device_of(0) == _device_of("cuda:0") == torch.device("cuda", 0)
    assert _device_of(2) == _device_of(torch.device("cuda", 2)) == torch.device("cuda", 2)
    with pytest.raises(ValueError, match="CUDA device"):
        IQPagedCache(1, 1, 1, device="cpu")
