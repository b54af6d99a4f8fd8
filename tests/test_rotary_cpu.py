"""Rotary positions without a GPU: frequencies against the oracle, and refusals.
Device pointers are made up and never followed."""
import ctypes

import numpy as np
import pytest

from oracle import rotary
from test_paged_cpu import CAPACITY, CUDA, INVALID, L, UNSUPPORTED, Fake, ints  # noqa: F401

A = 0x20000000  # a made-up device address


def frequencies(L, rd, base=10000.0, scaling=0, factor=1.0, original=0.0, low=0.0, high=0.0):
    f, a = np.zeros(128), ctypes.c_double()
    st = L.iq_rotary_frequencies(rd, base, scaling, factor, original, low, high, f.ctypes.data, ctypes.byref(a))
    return st, f[: max(rd, 0) // 2], a.value


@pytest.mark.parametrize("rd", [16, 64, 96, 128, 240, 256])
@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn", "banded"])
@pytest.mark.parametrize("base,factor,original", [(10000.0, 8.0, 4096), (1e7, 40.0, 32768), (500000.0, 1.0, 64)])
def test_frequencies(L, rd, scaling, base, factor, original):  # noqa: F811
    from rotated_bit_quantized_gb300 import rotary_frequencies
    f, amplitude = rotary_frequencies(rd, base, scaling, factor, original)
    lo, hi = {"yarn": (1, 32), "banded": (1, 4)}.get(scaling, (0, 0))
    want = [rotary.frequency(i, rd, base, scaling, factor, original, lo, hi) for i in range(rd // 2)]
    # powers and logarithms of the two libraries: a few units of the last place
    assert f == pytest.approx(want, rel=1e-14, abs=0)
    assert amplitude == (pytest.approx(1 + 0.1 * np.log(factor)) if scaling == "yarn" else 1.0)


def test_frequency_refusals(L):  # noqa: F811
    assert frequencies(L, 64)[0] == 0
    for rd in (0, -16, 8, 40, 272):
        assert frequencies(L, rd)[0] == UNSUPPORTED, rd
    nan, inf = float("nan"), float("inf")
    for kw in (dict(base=1.0), dict(base=nan), dict(base=inf), dict(scaling=5), dict(scaling=-1), dict(scaling=1, factor=0.5),
               dict(scaling=2, factor=nan), dict(scaling=3, factor=2, original=0, low=1, high=32), dict(scaling=3, factor=2, original=64, low=0, high=32),
               dict(scaling=4, factor=2, original=64, low=4, high=4), dict(scaling=4, factor=2, original=64, low=1, high=inf), dict(scaling=4, factor=2, original=nan, low=1, high=4)):
        assert frequencies(L, 64, **kw)[0] == INVALID, kw
    assert L.iq_rotary_frequencies(64, 1e4, 0, 1, 0, 0, 0, None, None) == INVALID


def test_turns_refusals(L):  # noqa: F811
    f = np.ones(128)
    for pairs, at, freq in ((0, A, f), (129, A, f), (8, 0, f), (8, A + 4, f), (2, A, np.array([1.0, np.nan])), (2, A, np.array([np.inf, 1.0]))):
        assert L.iq_rotary_turns(freq.ctypes.data, pairs, at, None) == INVALID, (pairs, at)
    assert L.iq_rotary_turns(None, 8, A, None) == INVALID


def desc(rd=64, interleaved=0, amplitude=1.0, eps=1e-6, turns=A, qw=0, kw=0):
    from rotated_bit_quantized_gb300._abi import IQRotaryDesc
    return ctypes.byref(IQRotaryDesc(rd, interleaved, amplitude, eps, turns, qw, kw))


def rows(at=A, entry=1 << 20, head=256, row=4096):
    from rotated_bit_quantized_gb300._abi import IQRows
    return ctypes.byref(IQRows(at, entry, head, row))


OUT_Q, OUT_K = 1 << 40, 1 << 41  # far from the inputs


def apply(L, d=None, dtype=0, q=None, qh=4, k=None, kh=2, entries=3, n=5, start=None, positions=None, q_out=OUT_Q, k_out=OUT_K):
    return L.iq_rotary_apply(d or desc(), dtype, q or rows(), qh, k or rows(), kh, entries, n, ints(start), 0 if start is None else len(start), positions, q_out, k_out, None)


BAD_PLANS = [(dict(rd=8), UNSUPPORTED), (dict(rd=-16), UNSUPPORTED), (dict(rd=272), UNSUPPORTED), (dict(interleaved=2), INVALID), (dict(turns=0), INVALID),
             (dict(turns=A + 4), INVALID), (dict(amplitude=float("inf")), INVALID), (dict(qw=A + 8), INVALID), (dict(kw=A, eps=0.0), INVALID),
             (dict(qw=A, eps=float("nan")), INVALID), (dict(qw=A, eps=1e-31), INVALID), (dict(qw=A, eps=float("inf")), INVALID)]


def test_apply_refusals(L):  # noqa: F811
    for kw, want in BAD_PLANS:
        assert apply(L, desc(**kw)) == want, kw
    assert L.iq_rotary_apply(None, 0, rows(), 1, rows(), 1, 1, 1, None, 0, None, OUT_Q, OUT_K, None) == INVALID
    for kw in (dict(dtype=2), dict(qh=-1), dict(kh=-1), dict(entries=-1), dict(n=-1), dict(entries=257), dict(start=[0, 1, 2], positions=A), dict(start=[0, 1]), dict(start=[0] * 4),
               dict(positions=A + 2), dict(q=rows(at=A + 8)), dict(q=rows(row=4100)), dict(k=rows(head=252)), dict(k=rows(entry=-4096)), dict(q=rows(row=1 << 41)),
               dict(q=rows(at=0)), dict(q_out=0), dict(k_out=0), dict(q_out=OUT_Q + 8), dict(q_out=A), dict(k_out=A + 4096),
               dict(q_out=OUT_K - 16), dict(k_out=OUT_Q + 4 * 3 * 5 * 512 - 16)):
        assert apply(L, **kw) == INVALID, kw
    assert apply(L, entries=256, n=1 << 22) == UNSUPPORTED
    assert apply(L, qh=(1 << 16) + 1) == UNSUPPORTED
    assert L.iq_rotary_apply(desc(), 0, None, 4, rows(), 2, 3, 5, None, 0, None, OUT_Q, OUT_K, None) == INVALID
    assert L.iq_rotary_apply(desc(), 0, rows(), 4, rows(), 2, 3, 5, None, 1, None, OUT_Q, OUT_K, None) == INVALID
    # nothing to do, whatever the pointers are
    assert apply(L, entries=0) == 0 and apply(L, n=0, q_out=0) == 0 and apply(L, qh=0, kh=0, q_out=0, k_out=0) == 0


def append(L, f, d=None, q=None, qh=4, k=None, v=None, n=5, slots=None, counts=None, entries=3, positions=None, q_out=OUT_Q):  # noqa: F811
    return L.iq_paged_append_rotary(f.p, d or desc(), q or rows(), qh, k or rows(), v or rows(), n, ints(slots), ints(counts), entries, positions, q_out, None)


def test_append_refusals_change_nothing(L):  # noqa: F811
    f = Fake(L)
    f.hold(0, [0, 1], 100)
    f.hold(1, [0, 1], 100)
    before = f.state()
    for kw, want in BAD_PLANS:
        assert append(L, f, desc(**kw)) == want, kw
    assert L.iq_paged_append_rotary(f.p, None, rows(), 4, rows(), rows(), 1, None, None, 1, None, OUT_Q, None) == INVALID
    assert L.iq_paged_append_rotary(None, desc(), rows(), 4, rows(), rows(), 1, None, None, 1, None, OUT_Q, None) == INVALID
    for kw in (dict(qh=-1), dict(n=-1), dict(entries=5), dict(slots=[0, 0, 1]), dict(slots=[0, 1, 4]), dict(counts=[1, 6, 0]), dict(counts=[-1, 0, 0]),
               dict(positions=A + 1), dict(k=rows(at=0)), dict(v=rows(at=A + 4)), dict(k=rows(row=4097)), dict(v=rows(entry=-8)), dict(q=rows(head=100)),
               dict(q_out=0), dict(q_out=OUT_Q + 2), dict(q_out=A)):
        assert append(L, f, **kw) == INVALID, kw
    assert append(L, f, n=1000) == CAPACITY
    assert append(L, f, qh=(1 << 14) + 1) == UNSUPPORTED
    assert f.state() == before


def test_append_undone_where_the_launch_fails(L):  # noqa: F811
    f = Fake(L)
    f.hold(0, [0, 1], 100)
    f.hold(1, [0, 1], 100)
    before = f.state()
    L.iq_paged_debug_fail(0)
    assert append(L, f, n=40) == CUDA
    L.iq_paged_debug_fail(-1)
    assert f.state() == before


def test_binding_refusals():
    import torch

    from rotated_bit_quantized_gb300 import IQRotary, rotary_frequencies
    with pytest.raises(ValueError):
        rotary_frequencies(64, scaling="other")
    for kw in (dict(head_dim=128), dict(rotary_dim=24), dict(rotary_dim=-16), dict(rotary_dim=32, frequencies=[1.0] * 15), dict(rotary_dim=16, frequencies=[float("nan")] * 8),
               dict(amplitude=float("inf")), dict(q_norm=torch.ones(256), eps=0.0), dict(k_norm=torch.ones(255)), dict(q_norm=torch.ones(256, dtype=torch.int32))):
        with pytest.raises(ValueError):
            IQRotary(**kw)


def test_rows_whose_span_passes_64_bits(L):  # noqa: F811
    """Strides within their limit whose product with the rows is not an address: refused, not wrapped round."""
    wide = (1 << 23) + 1  # 2^40 elements of 2 bytes, times 2^23: 2^64
    for kw in (dict(q=rows(row=1 << 40)), dict(k=rows(row=1 << 40))):
        assert apply(L, n=wide, **kw) == INVALID, kw
    assert apply(L, dtype=1, n=(1 << 22) + 1, q=rows(row=1 << 40)) == INVALID
    assert apply(L, n=(1 << 22) + 1, entries=3, q=rows(entry=1 << 40, row=1 << 40)) == INVALID
    f = Fake(L, pages=1 << 20, max_pages=1 << 18)
    before = f.state()
    for kw in (dict(q=rows(row=1 << 40)), dict(k=rows(row=1 << 40)), dict(v=rows(row=1 << 40))):
        assert append(L, f, n=wide, entries=1, **kw) == INVALID, kw
    assert f.state() == before


def test_a_plan_is_for_a_cuda_device():
    """A name of another kind of device is refused, not taken for the current CUDA device."""
    import torch

    from rotated_bit_quantized_gb300 import IQRotary
    for device in ("cpu", torch.device("cpu"), "meta"):
        with pytest.raises(ValueError):
            IQRotary(rotary_dim=0, device=device)


@pytest.mark.parametrize("captured", [0, 1])
def test_a_plan_waits_where_its_own_device_captures_nothing(captured, monkeypatch):
    """Whether the plan's device is capturing is asked of that device, whichever is current."""
    import torch

    from rotated_bit_quantized_gb300 import rotary as r
    current, waited = [0], []

    class On:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.prev, current[0] = current[0], self.index

        def __exit__(self, *_):
            current[0] = self.prev

    class Stream:
        def synchronize(self):
            waited.append(True)
    monkeypatch.setattr(r, "_OnDevice", On)
    monkeypatch.setattr(r, "_capturing", lambda: current[0] == captured)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream())
    r.IQRotary(rotary_dim=0, device="cuda:1")
    assert bool(waited) == (captured != 1) and current == [0]
