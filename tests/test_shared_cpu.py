"""Attention of shared pages without a GPU: workspaces, refusals, and appends undone.  Device pointers are made up and never followed."""
import ctypes

import numpy as np
import pytest

from test_paged_cpu import CAPACITY, CUDA, INVALID, L, P, UNSUPPORTED, WORKSPACE, Fake, ints  # noqa: F401


def workspace(L, f, Hq, n, k, shared):  # noqa: F811
    b = ctypes.c_size_t()
    st = (L.iq_paged_attend_shared_workspace if shared else L.iq_paged_attend_workspace)(f.p, Hq, n, k, ctypes.byref(b))
    return st, b.value


def attend(f, Hq=4, n=1, slots=None, counts=None, k=4, scale=0.1, causal=1, window=0, sinks=0, out_f32=0, q=P, out=P, ws=P, nbytes=1 << 40):
    return f.L.iq_paged_attend_shared(f.p, q, Hq, n, ints(slots), ints(counts), k, scale, causal, window, sinks, out, out_f32, ws, nbytes, None)


def test_workspace(L):  # noqa: F811
    f = Fake(L)
    for Hq, n, k in ((4, 1, 4), (16, 3, 2), (2, 64, 4)):
        st, plain = workspace(L, f, Hq, n, k, False)
        st2, shared = workspace(L, f, Hq, n, k, True)
        assert st == st2 == 0 and shared >= plain
        # four levels of every row's partial results, the cut queries
        assert shared >= Hq * n * k * (4 * 1032 + 516)
    for Hq, n, k in ((4, 65, 4), (4, 1, 1), (4, 0, 4), (4, 1, 0)):  # more than 128 rows of a slot, one slot, nothing
        assert workspace(L, f, Hq, n, k, False) == workspace(L, f, Hq, n, k, True)
    for Hq, n, k, want in ((3, 1, 4, UNSUPPORTED), (4, -1, 4, INVALID), (4, 1, 257, INVALID), (130, 1, 4, UNSUPPORTED)):
        assert workspace(L, f, Hq, n, k, True)[0] == want
    assert L.iq_paged_attend_shared_workspace(f.p, 4, 1, 4, None) == INVALID


def test_refusals(L):  # noqa: F811
    f = Fake(L)
    f.hold(0, [0, 1], 100)
    f.hold(1, [0, 1], 100)
    need = workspace(L, f, 4, 1, 4, True)[1]
    for kw, want in ((dict(q=None), INVALID), (dict(out=None), INVALID), (dict(q=ctypes.c_void_p(8)), INVALID), (dict(causal=2), INVALID), (dict(window=-1), INVALID),
                     (dict(window=3, causal=0), INVALID), (dict(sinks=1), INVALID), (dict(scale=float("inf")), INVALID), (dict(out_f32=2), INVALID),
                     (dict(slots=[0, 1, 2, 4]), INVALID), (dict(counts=[0, 0, 2, 0]), INVALID), (dict(k=5), INVALID), (dict(Hq=3), UNSUPPORTED), (dict(ws=None), WORKSPACE),
                     (dict(nbytes=need - 1), WORKSPACE), (dict(ws=ctypes.c_void_p(0x20000010)), WORKSPACE)):
        assert attend(f, **kw) == want, kw
    assert attend(f, n=0) == 0 and attend(f, k=0) == 0


def test_append_attend_refuses_before_it_appends(L):  # noqa: F811
    f = Fake(L)
    f.hold(0, [0, 1], 100)
    f.hold(1, [0, 1], 100)
    before = f.state()
    need = workspace(L, f, 4, 1, 4, True)[1]

    def call(n=1, Hq=4, nq=1, counts=None, sinks=0, ws=P, nbytes=need, keys=P, slots=None):
        return L.iq_paged_append_attend_shared(f.p, keys, P, n, P, Hq, nq, ints(slots), ints(counts), 4, 0.1, 1, 0, sinks, P, 0, ws, nbytes, None)
    for kw, want in ((dict(keys=None), INVALID), (dict(n=-1), INVALID), (dict(n=2, counts=[1, 1, 1, 1]), INVALID), (dict(sinks=1), INVALID), (dict(Hq=3), UNSUPPORTED),
                     (dict(nbytes=need - 1), WORKSPACE), (dict(ws=None), WORKSPACE), (dict(n=10000), CAPACITY), (dict(slots=[0, 1, 1, 2]), INVALID)):
        assert call(**kw) == want, kw
        assert f.state() == before
    L.iq_paged_debug_fail(0)
    assert call() == CUDA and f.state() == before
    L.iq_paged_debug_fail(-1)


@pytest.mark.parametrize("slots", [2, 32])
def test_plans_of_any_table(L, slots):  # noqa: F811
    """Tables of all shapes are planned up to the first launch or tensor map, which there is no GPU for: an error, not a crash."""
    rng = np.random.default_rng(slots)
    for case in range(40):
        f = Fake(L, slots=slots, pages=4000, max_pages=60)
        for s in range(slots):  # random trees: some earlier slot's pages, then some of its own
            other = int(rng.integers(s)) if s and rng.random() < 0.8 else s
            row = [] if other == s else [int(p) for p in f.table[other, : rng.integers(0, -(-int(f.lens[other]) // 64) + 1)]][:50]
            row += list(range(60 * s, 60 * s + int(rng.integers(0, 9))))
            f.hold(s, row, int(rng.integers(max(0, 64 * len(row) - 63), 64 * len(row) + 1)) if row else 0)
        st = attend(f, Hq=16, n=int(rng.integers(1, 9)), k=slots, window=int(rng.integers(0, 2) * rng.integers(0, 3000)))
        assert st in (0, CUDA)
