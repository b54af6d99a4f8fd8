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


def plan(f, Hq, n, slots=None, counts=None, k=4, causal=1, window=0, sinks=0, forced=1):
    """The plan of a call: its header, nodes and entries as named numbers."""
    from rotated_bit_quantized_gb300._abi import IQ_PLAN_WORDS
    w = np.zeros(IQ_PLAN_WORDS, dtype=np.int32)
    assert f.L.iq_paged_debug_plan(f.p, Hq, n, ints(slots), ints(counts), k, causal, window, sinks, forced, w.ctypes.data) == 0
    head = dict(zip(("nodes", "leaves", "entries", "rows", "wide", "narrow", "wide_cost", "narrow_cost", "wide_total", "narrow_total", "narrow_rows", "parts"), w.tolist()))
    names = ("slot", "parent", "end_page", "row0", "n", "part0", "cum", "tiles", "base", "sinks", "skip", "p_lo", "p_hi")
    nodes = [dict(zip(names, w[12 + 13 * i: 25 + 13 * i].tolist())) for i in range(head["nodes"])]
    at = 12 + 13 * head["nodes"]
    return head, nodes, [dict(zip(("place", "lowest", "row0", "pos0"), w[at + 4 * i: at + 4 * i + 4].tolist())) for i in range(head["entries"])]


def check_plan(f, Hq, n, slots, counts, k, causal, window, sinks, forced):
    """Every key that a row sees is in exactly one tile of the nodes above it, of pages that its own slot holds; rows, partial
    results and slots of the ranges lie side by side without a gap, and within the workspace."""
    head, nodes, entries = plan(f, Hq, n, slots, counts, k, causal, window, sinks, forced)
    if not nodes:
        return False
    heads, rep = f.d.kv_heads, Hq // f.d.kv_heads
    ids, cnt = list(range(k)) if slots is None else slots, [n] * k if counts is None else counts
    live = [i for i in range(k) if cnt[i] and f.lens[ids[i]]]
    assert sorted(e["place"] for e in entries) == live and head["rows"] == sum(cnt[i] * rep for i in live)
    tiles = [[x["base"] + (j if j < x["sinks"] else j + x["skip"]) for j in range(x["tiles"])] for x in nodes]
    assert all(len(t) > 0 and len(set(t)) == len(t) for t in tiles) and len(nodes) <= 320
    rows, under = 0, [[] for _ in nodes]
    for e in entries:
        i = e["place"]
        slot, own = ids[i], cnt[i] * rep
        length = int(f.lens[slot])
        pages = f.table[slot, : -(-length // 64)]
        assert e["row0"] == rows
        rows += own
        path, x = [], e["lowest"]
        while x >= 0:
            path.append(x)
            x = nodes[x]["parent"]
        assert 1 <= len(path) <= 4
        seen = [t for x in path for t in tiles[x]]
        assert len(seen) == len(set(seen))  # once
        for x in path:
            node = nodes[x]
            assert node["row0"] <= e["row0"] and e["row0"] + own <= node["row0"] + node["n"]
            under[x].append(own)
            holder = f.table[node["slot"]]
            for t in tiles[x]:
                for page in (2 * t, 2 * t + 1):
                    if page < len(pages):  # what the node reads there is this slot's too
                        assert page <= node["end_page"] and holder[page] == pages[page]
        first = length - cnt[i] if causal else length - 1
        assert e["pos0"] == first
        wanted = set()
        for j in range(cnt[i]):
            at = first + j if causal else length - 1
            for x in path:
                assert nodes[x]["p_lo"] <= at <= nodes[x]["p_hi"]
            if at < 0:
                continue
            low = max(0, at - window + 1) if 0 < window < max(f.lens[s] for s in ids) else 0
            wanted |= set(range(low // 128, at // 128 + 1)) | (set(range((min(sinks, low) + 127) // 128)) if low else set())
        assert wanted <= set(seen)
    assert rows == head["rows"]
    part = 0
    for kind, (a, b) in enumerate(((0, head["leaves"]), (head["leaves"], len(nodes)))):
        total, cost = 0, head["narrow_cost" if kind else "wide_cost"]
        for x in range(a, b):
            node = nodes[x]
            assert sum(under[x]) == node["n"] and node["cum"] == total
            assert -1 <= node["parent"] < head["leaves"] and (not kind or len(under[x]) == 1 and node["n"] <= head["narrow_rows"])
            part += heads * node["n"]
            total += heads * -(-node["n"] // 128) * (node["tiles"] + cost)
        assert head["narrow_total" if kind else "wide_total"] == total
        grid = head["narrow" if kind else "wide"]
        assert grid == 0 if total == 0 else 1 <= grid <= sum(heads * -(-nodes[x]["n"] // 128) * nodes[x]["tiles"] for x in range(a, b))
    at = 0
    for x in sorted(nodes, key=lambda x: x["part0"]):
        assert x["part0"] == at
        at += heads * x["n"]
    assert at == part
    assert head["parts"] == part + 128 * head["wide"] + head["narrow_rows"] * head["narrow"]
    assert head["parts"] * 1032 + head["rows"] * (8 + heads * (512 + 4 + 64)) <= workspace(f.L, f, Hq, n, k, True)[1]
    return True


@pytest.mark.parametrize("slots", [2, 7, 40, 250])
def test_plans_read_every_key_once(L, slots):  # noqa: F811
    rng = np.random.default_rng(slots)
    planned = faster = 0
    for case in range(60 if slots < 250 else 20):
        f = Fake(L, slots=slots, heads=int(rng.choice([1, 2, 8])), pages=slots * 60, max_pages=60)
        wide = rng.random() < 0.3  # long common prompts, of which sharing is the faster way
        for s in range(slots):
            other = int(rng.integers(s)) if s and rng.random() < (0.95 if wide else 0.8) else s
            held = -(-int(f.lens[other]) // 64) if other != s else 0
            row = [int(p) for p in f.table[other, : held if wide else rng.integers(0, held + 1)]][:50]
            full = len(row) == held and rng.random() < 0.5  # goes on or ends in the shared last page
            fresh = 0 if full else int(rng.integers(0, 9)) + (40 if wide and not row else 0)
            row += list(range(60 * s, 60 * s + fresh))
            f.hold(s, row, int(rng.integers(max(0, 64 * len(row) - 63), 64 * len(row) + 1)) if row else 0)
        listed = rng.integers(0, slots, slots).tolist() if rng.random() < 0.3 else None  # some twice
        n = int(rng.integers(1, 5))
        counts = rng.integers(0, n + 1, slots).tolist() if rng.random() < 0.3 else None
        causal = int(rng.random() < 0.8)
        window = int(rng.integers(1, 3000)) if causal and rng.random() < 0.5 else 0
        sinks = int(rng.choice([0, 1, 4, 130, 700])) if window else 0
        args = (f.d.kv_heads * int(rng.choice([1, 3, 8])), n, listed, counts, slots, causal, window, sinks)
        planned += check_plan(f, *args, 1)
        faster += check_plan(f, *args, 0)
    assert planned > 10 and faster >= (0 if slots < 7 else 1)


def test_plans_of_many_groups(L):  # noqa: F811
    """More shared runs than there is room for: the later ones' slots read their own."""
    f = Fake(L, slots=240, heads=2, pages=240 * 12, max_pages=12)
    for s in range(240):
        g = s // 3
        f.hold(s, list(range(12 * 3 * g, 12 * 3 * g + 9)) + [36 * g + 9 + s % 3], 64 * 9 + 5)
    assert check_plan(f, 8, 1, None, None, 240, 1, 0, 0, 1)
    head, nodes, _ = plan(f, 8, 1, k=240)
    assert sum(x["n"] == 12 for x in nodes) == 64 and len(nodes) == 64 + 240


def test_plan_refusals(L):  # noqa: F811
    f = Fake(L)
    w = np.zeros(8000, dtype=np.int32)
    call = lambda Hq=4, n=1, counts=None, k=4, causal=1, window=0, sinks=0, at=w.ctypes.data: L.iq_paged_debug_plan(f.p, Hq, n, None, ints(counts), k, causal, window, sinks, 1, at)  # noqa: E731
    for kw, want in ((dict(Hq=3), UNSUPPORTED), (dict(n=-1), INVALID), (dict(k=5), INVALID), (dict(causal=2), INVALID), (dict(window=-1), INVALID), (dict(sinks=1), INVALID),
                     (dict(counts=[2, 0, 0, 0]), INVALID), (dict(at=None), INVALID)):
        assert call(**kw) == want, kw
    assert call() == 0 and call(n=0) == 0 and call(k=0) == 0 and w[0] == 0
    assert L.iq_paged_debug_plan(None, 4, 1, None, None, 4, 1, 0, 0, 1, w.ctypes.data) == INVALID


def test_plans_of_a_pool_that_is_16_byte_aligned(L):  # noqa: F811
    f = Fake(L, base=0x10000010)
    for s in range(4):
        f.hold(s, [0, 1, 2 + s], 150)
    assert check_plan(f, 8, 1, None, None, 4, 1, 0, 0, 1)
