"""Attention of slots that share pages, each shared page multiplied once: against the oracle, within the bounds of the
attention that reads every slot's pages apart."""
import numpy as np
import pytest
import torch

from oracle import paged
from test_gpu_paged import bounds, f64, pair, put, rows

pytestmark = pytest.mark.gpu


def shared(c, q, **kw):
    """Shared wherever there are pages to share, however little is gained."""
    from rotated_bit_quantized_gb300 import _abi
    assert _abi.lib().iq_paged_debug_share() == 0
    return c.attend(q, shared=True, **kw)


def check(c, o, q, out_dtype=torch.float32, slots=None, counts=None, scale=1 / 16, **kw):
    out = shared(c, q.cuda(), scale=scale, slots=slots, counts=counts, out_dtype=out_dtype, **kw)
    assert out.dtype == out_dtype and out.shape == q.shape
    res = paged.attend(o, f64(q), scale, slots, counts, **kw)
    got, live = f64(out), ~np.isnan(res[0])
    tol, d = bounds(res, out_dtype == torch.float32), np.abs(got - res[0])
    assert np.isfinite(got).all()
    assert (d[live] <= tol[live]).all(), (d[live] / tol[live]).max()
    if counts is not None:
        assert (got[~live] == 0).all()
    score = np.linalg.norm((2 * (2.0**-17 + 2.0**-16) * res[3] * res[1])[live])
    assert np.linalg.norm(d[live]) <= 2.0**-8 * np.linalg.norm(res[0][live]) + score + 1e-30
    assert c.device_status() == 0
    return out


def tree(H, common, branch, tails, groups=1, seed=1, outliers=True):
    """`groups` branches of one prompt, and len(tails) paths of each (the tails' lengths)."""
    paths = len(tails) // groups
    slots = len(tails)
    c, o = pair(slots, H, (common + 63) // 64 + 1 + groups * ((branch + 127) // 64) + sum(2 + t // 64 for t in tails), common + branch + max(tails) + 1)
    put(c, o, rows(seed, 1, H, common, outliers), rows(seed + 1, 1, H, common), [0])
    leaders = list(range(0, slots, paths))
    for x in (c, o):
        x.fork([0] * (groups - 1), leaders[1:])
    if branch:
        put(c, o, rows(seed + 2, groups, H, branch, outliers), rows(seed + 3, groups, H, branch), leaders)
    others = [s for s in range(slots) if s not in leaders]
    for x in (c, o):
        x.fork([s - s % paths for s in others], others)
    if max(tails):
        put(c, o, rows(seed + 4, slots, H, max(tails), outliers), rows(seed + 5, slots, H, max(tails)), list(range(slots)), list(tails))
    return c, o


@pytest.mark.parametrize("H,Hq,n", [(1, 1, 1), (2, 16, 1), (2, 6, 3), (4, 4, 1), (1, 64, 2), (1, 5, 25), (3, 24, 4)])
@pytest.mark.parametrize("paths,common", [(2, 1024), (4, 513), (33, 320), (17, 2000)])
def test_paths_of_one_prompt(H, Hq, n, paths, common):
    c, o = tree(H, common, 0, [1 + (37 * b) % 150 + n for b in range(paths)])
    check(c, o, rows(9, paths, Hq, n))


@pytest.mark.parametrize("common,branch,tail,groups,paths", [(640, 300, 70, 3, 5), (64, 1000, 1, 2, 9), (1, 800, 130, 4, 3), (129, 127, 129, 5, 4), (2049, 65, 63, 2, 20)])
@pytest.mark.parametrize("n", [1, 4])
def test_branches_of_a_prompt(common, branch, tail, groups, paths, n):
    c, o = tree(2, common, branch, [tail + (11 * b) % 9 + n for b in range(groups * paths)], groups)
    check(c, o, rows(9, groups * paths, 12, n), torch.bfloat16)
    check(c, o, rows(10, groups * paths, 12, n))


@pytest.mark.parametrize("common", [1, 63, 64, 127, 128, 191, 700, 1000])
@pytest.mark.parametrize("n", [1, 5])
def test_forks_that_nobody_has_appended_to(common, n):
    """The last, partly full page is shared too; of several queries only the last see all of it, some of one token's none."""
    c, o = tree(2, common, 0, [0] * 6)
    check(c, o, rows(9, 6, 4, n))


def test_slots_trimmed_inside_a_shared_page():
    c, o = tree(2, 1000, 0, [0] * 9)
    for x in (c, o):
        x.trim([0, 1, 30, 41, 100, 500, 999, 1000, 3], list(range(9)))
    q = rows(9, 9, 8, 2)
    check(c, o, q)
    put(c, o, rows(5, 9, 2, 2), rows(6, 9, 2, 2))
    check(c, o, q)


@pytest.mark.parametrize("window,sinks", [(1, 0), (100, 0), (100, 7), (128, 128), (700, 1), (900, 300), (5000, 3)])
@pytest.mark.parametrize("n", [1, 4])
def test_windows(window, sinks, n):
    c, o = tree(2, 1100, 500, [n + (53 * b) % 400 for b in range(12)], 2)
    check(c, o, rows(9, 12, 8, n), window=window, sinks=sinks)


def test_queries_that_see_every_key():
    c, o = tree(2, 700, 200, [1 + (53 * b) % 400 for b in range(12)], 2)
    check(c, o, rows(9, 12, 8, 3), causal=False)


def test_lists_of_slots_counts_and_empty_slots():
    c, o = tree(2, 600, 100, [3 + (53 * b) % 200 for b in range(12)], 2)
    for x in (c, o):
        x.free([4, 7])
        x.trim([10**6], [5])
    put(c, o, rows(5, 1, 2, 2), rows(6, 1, 2, 2), [5])  # a short slot of its own: two tokens, more queries than these
    slots = [11, 4, 0, 5, 3, 3, 7, 8, 2, 0, 9]
    q = rows(9, len(slots), 8, 5)
    check(c, o, q, slots=slots)
    counts = [5, 5, 0, 4, 1, 5, 0, 2, 3, 5, 1]
    check(c, o, q, slots=slots, counts=counts)
    out = torch.full((len(slots), 8, 5, 256), 7.0, device="cuda")
    shared(c, q.cuda(), slots=slots, counts=counts, out=out)
    for i, n in enumerate(counts):
        assert (out[i, :, n:] == 7).all() and not (out[i, :, :n] == 7).any()


def test_deep_and_wide_trees():
    """More levels than are told apart, and more branches than there is room for."""
    c, o = pair(40, 1, 700, 3000)
    put(c, o, rows(1, 1, 1, 300), rows(2, 1, 1, 300), [0])
    live = 1
    for level in range(5):  # every slot is forked, then goes on by itself
        for x in (c, o):
            x.fork(list(range(live)), list(range(live, 2 * live)))
        live *= 2
        put(c, o, rows(3 + level, live, 1, 270), rows(20 + level, live, 1, 270), list(range(live)))
    check(c, o, rows(9, 32, 4, 1))
    check(c, o, rows(9, 40, 4, 2))
    c, o = pair(240, 1, 1200, 700)
    firsts = list(range(0, 240, 3))
    put(c, o, rows(1, 80, 1, 640), rows(2, 80, 1, 640), firsts)
    for x in (c, o):
        x.fork([s for s in firsts for _ in (0, 1)], [s + i for s in firsts for i in (1, 2)])
    put(c, o, rows(3, 240, 1, 3), rows(4, 240, 1, 3))
    check(c, o, rows(9, 240, 8, 1))


def test_many_slots_and_rows():
    c, o = tree(2, 200, 0, [1 + b % 3 for b in range(256)], outliers=False)
    check(c, o, rows(9, 256, 16, 1))
    check(c, o, rows(9, 256, 2, 3), torch.bfloat16)


@pytest.mark.parametrize("Hq,n", [(8, 1), (16, 2), (32, 2)])  # of 4, 16 and 32 rows a head
@pytest.mark.parametrize("shift", [0, 1])
def test_leaves_of_few_tiles_in_turn(Hq, n, shift):
    """Several leaves a CTA, of one to six tiles, odd and even numbers after one another; heavy keys in one tile of some."""
    H, tails = 2, [1 + n + 128 * ((5 * b + b // 7 + shift) % 6) + (37 * b) % 120 for b in range(170)]
    c, o = tree(H, 256, 0, tails, outliers=False)
    heavy = list(range(0, 170, 3))
    for x in (c, o):
        x.trim([int(256 + max(1, t - 100)) for t in tails], list(range(170)))
    put(c, o, 60 * rows(7, len(heavy), H, n), rows(8, len(heavy), H, n), heavy)
    check(c, o, rows(9, 170, Hq, n))


@pytest.mark.parametrize("scale", [-1 / 16, 0.0, 2.0, 1e-6])
def test_scales(scale):
    c, o = tree(2, 700, 0, [1 + (53 * b) % 200 for b in range(8)])
    check(c, o, rows(9, 8, 8, 1), scale=scale)


def test_queries_that_are_not_finite_keep_to_themselves():
    c, o = tree(2, 700, 0, [1 + (53 * b) % 200 for b in range(8)])
    q = rows(9, 8, 8, 2)
    bad = q.clone()
    bad[2, 3, 1, 17], bad[5, 0, 0, 200], bad[7, 7, 1, 0] = float("nan"), float("inf"), -float("inf")
    good, got, apart = shared(c, q.cuda()), shared(c, bad.cuda()), c.attend(bad.cuda())
    touched = ~torch.isfinite(bad).all(-1).cuda()
    assert torch.equal(got[~touched], good[~touched])
    assert torch.isnan(apart[touched]).all() and torch.isnan(got[touched]).all()


def test_one_heavy_key_among_many():
    """What many small weights leave next to a heavy key of the shared part, and of a path's own."""
    for heavy in (5, 1290):
        c, o = pair(6, 1, 140, 1400)
        k, v = rows(1, 1, 1, 1280), rows(2, 1, 1, 1280)
        k2, v2 = rows(3, 6, 1, 40), rows(4, 6, 1, 40)
        k[..., 0] = k2[..., 0] = 0
        (k if heavy < 1280 else k2)[:, :, heavy % 1280, 0] = 90
        (v if heavy < 1280 else v2)[:, :, heavy % 1280] = 0
        put(c, o, k, v, [0])
        for x in (c, o):
            x.fork([0] * 5, [1, 2, 3, 4, 5])
        put(c, o, k2, v2)
        q = 0.05 * rows(9, 6, 4, 1)
        q[..., 0] = 1.3
        check(c, o, q)


def test_same_results_every_time_and_on_every_path():
    c, _ = tree(2, 3000, 700, [1 + (53 * b) % 200 for b in range(20)], 4)
    q = rows(9, 20, 16, 1).cuda()
    first = shared(c, q)
    for _ in range(10):
        assert torch.equal(shared(c, q), first)
    many = rows(9, 20, 16, 17).cuda()  # 136 rows of a slot: the ordinary kernels
    assert torch.equal(c.attend(many, shared=True), c.attend(many))
    alone = rows(9, 1, 16, 1).cuda()
    assert torch.equal(c.attend(alone, slots=[3], shared=True), c.attend(alone, slots=[3]))
    small = c.compact()
    assert torch.equal(shared(small, q), first)
    little, _ = tree(2, 70, 0, [1, 2])  # nothing to gain: as without
    q = rows(9, 2, 16, 1).cuda()
    assert torch.equal(little.attend(q, shared=True), little.attend(q))


@pytest.mark.parametrize("paths,common,n", [(2, 512, 1), (8, 2048, 1), (32, 4096, 1), (32, 1024, 4), (5, 3000, 13)])
def test_whichever_way_is_taken(paths, common, n):
    c, o = tree(2, common, 0, [n + (37 * b) % 90 for b in range(paths)])
    q = rows(9, paths, 16, n)
    way = c.attend(q.cuda(), shared=True, out_dtype=torch.float32)
    either = [c.attend(q.cuda(), out_dtype=torch.float32), check(c, o, q)]
    assert any(torch.equal(way, e) for e in either)


def test_append_attend_as_two_calls():
    from rotated_bit_quantized_gb300 import _abi
    a, _ = tree(2, 900, 0, [5 + b for b in range(7)])
    b, _ = tree(2, 900, 0, [5 + b for b in range(7)])
    k, v, q = rows(5, 7, 2, 3).cuda(), rows(6, 7, 2, 3).cuda(), rows(9, 7, 8, 3).cuda()
    counts = [3, 0, 1, 2, 3, 3, 1]
    assert _abi.lib().iq_paged_debug_share() == 0
    x = a.append_attend(k, v, q, counts=counts, shared=True, window=600, sinks=2)
    b.append(k, v, counts=counts)
    assert torch.equal(x, shared(b, q, counts=counts, window=600, sinks=2))
    before = a.lens.tolist()
    with pytest.raises(_abi.IQError):
        a.append_attend(k, v, q, shared=True, sinks=1)
    assert a.lens.tolist() == before


def test_streams_and_graphs():
    c, o = tree(2, 1500, 0, [9 + b for b in range(9)])
    q = rows(9, 9, 8, 1).cuda()
    want = shared(c, q)
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs += [shared(c, q) for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in outs)
    graphs = []
    for s in streams[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            graphs.append((g, shared(c, q)))
    q2 = rows(19, 9, 8, 1).cuda()
    want2 = shared(c, q2)
    torch.cuda.synchronize()
    q.copy_(q2)
    torch.cuda.synchronize()
    for s, (g, _) in zip(streams, graphs):  # two at once
        with torch.cuda.stream(s):
            for _ in range(5):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, want2) for _, x in graphs)


def test_waits_run_out():
    from rotated_bit_quantized_gb300 import _abi
    c, o = tree(1, 1000, 0, [5] * 4)
    q = rows(9, 4, 4, 1)
    assert _abi.lib().iq_paged_debug_stall() == 0
    shared(c, q.cuda())
    assert c.device_status() & 0xB
    check(c, o, q)


def test_a_bad_page_is_told_and_read_as_another():
    from rotated_bit_quantized_gb300 import _abi
    c, o = tree(1, 1000, 0, [5] * 4)
    q = rows(9, 4, 4, 1).cuda()
    shared(c, q)
    torch.cuda.synchronize()
    keep = c.table.clone()
    c.table[:, 3] = 10**6
    shared(c, q)
    assert c.device_status() == _abi.IQ_STATUS_BAD_PAGE
    c.table.copy_(keep)
    check(c, o, rows(9, 4, 4, 1))


def test_a_decode_step_of_all_of_it():
    """Projections of forked paths: normed, turned and appended, then attended with the shared pages read once."""
    from rotated_bit_quantized_gb300 import IQPagedCache, IQRotary
    g = torch.Generator().manual_seed(1)
    rot = IQRotary(64, base=1e6, q_norm=0.1 * torch.randn(256, generator=g), k_norm=0.1 * torch.randn(256, generator=g), norm_offset=1.0)
    a, b = IQPagedCache(9, 2, 60), IQPagedCache(9, 2, 60)
    for c in (a, b):
        x = rows(1, 1, 1, 700 * 12).view(1, 700, 12, 256).transpose(1, 2).cuda()
        c.append_rotary(None, x[:, 8:10], x[:, 10:], rot, slots=[0])
        c.fork([0] * 8, range(1, 9))
    for step in range(4):
        x = rows(10 + step, 1, 1, 8 * 12).view(8, 1, 12, 256).transpose(1, 2).cuda()
        q = a.append_rotary(x[:, :8], x[:, 8:10], x[:, 10:], rot, slots=range(1, 9))
        one = shared(a, q, slots=range(1, 9), out_dtype=torch.float32)
        q2, k2 = rot.apply(x[:, :8], x[:, 8:10], positions=700 + step)
        assert torch.equal(q, q2)
        b.append(k2, x[:, 10:].contiguous(), slots=range(1, 9))
        two = b.attend(q2, slots=range(1, 9), out_dtype=torch.float32)
        # keys rounded once and twice differ by a code's step (2^-3) here and there, weights by 2^-8 twice
        assert (one - two).norm() <= 0.02 * two.norm()
        for i, p in enumerate(a.page_ids(1)[: 700 // 64]):
            assert (b.page_ids(1)[i] == p)
    assert a.device_status() == 0 and b.device_status() == 0


@pytest.mark.parametrize("paths,common,tail,Hq,n", [(6, 640, 90, 4, 1), (12, 1000, 300, 16, 2), (3, 513, 200, 32, 2), (40, 300, 20, 8, 5)])
def test_values_that_are_all_alike_come_back(paths, common, tail, Hq, n):
    """Weights are divided by the sum of the weights as they are held, so their own rounding cancels; what is left are the
    roundings of float32 sums of positive numbers, 2^-23 of the sum each: 16 a tile in the products (8 of them, cut inside and
    added), 34 and one a tile in the sums of weights, under 12 tiles: 240, and 16 for the joins and the division."""
    H = 2
    c, o = pair(paths, H, (common + 63) // 64 + paths * (2 + tail // 64), common + tail + 1)
    alike = torch.tensor([1.0, -1.5, 0.75, 2.0, -0.25, 0.875, -1.125, 1.75]).repeat(32).to(torch.bfloat16)
    put(c, o, rows(1, 1, H, common), alike.expand(1, H, common, 256), [0])
    for x in (c, o):
        x.fork([0] * (paths - 1), list(range(1, paths)))
    put(c, o, rows(2, paths, H, tail), alike.expand(paths, H, tail, 256))
    q = 3 * rows(9, paths, Hq, n).cuda()
    for out in (c.attend(q, out_dtype=torch.float32), shared(c, q, out_dtype=torch.float32)):
        assert (f64(out) / f64(alike) - 1).__abs__().max() <= 256 * 2.0**-23
    assert c.device_status() == 0


@pytest.mark.parametrize("Hq", [2, 8])  # of 4 and 16 rows a head
def test_turns_that_end_apart(Hq):
    """Two warpgroups take a leaf's tiles in turn and join their results: leaves of one to ten tiles, of which one
    warpgroup's keys hold references that move in every tile; the same from call to call."""
    H, n, paths = 1, 2, 60
    c, o = pair(paths, H, 2 + paths * 22, 256 + 1400)
    put(c, o, rows(1, 1, H, 256), rows(2, 1, H, 256), [0])
    for x in (c, o):
        x.fork([0] * (paths - 1), list(range(1, paths)))
    k = rows(3, paths, H, 1290)
    for t in range(1290):  # growing, in every other tile
        k[:, :, t] *= 1 + 10 * (t // 128) if (t // 128) % 2 else 1
    put(c, o, k, rows(4, paths, H, 1290), None, [n + (149 * b) % 1280 for b in range(paths)])
    q = rows(9, paths, Hq, n)
    first = check(c, o, q)
    for _ in range(30):
        assert torch.equal(shared(c, q.cuda(), out_dtype=torch.float32), first)


def forked(k, v, k2, v2, H=1):
    """Paths of one prompt (k, v) with rows of their own (k2, v2)."""
    paths, common, tail = k2.shape[0], k.shape[2], k2.shape[2]
    c, o = pair(paths, H, (common + 63) // 64 + paths * (2 + tail // 64), common + tail)
    put(c, o, k, v, [0])
    for x in (c, o):
        x.fork([0] * (paths - 1), list(range(1, paths)))
    put(c, o, k2, v2)
    return c, o


@pytest.mark.parametrize("n", [1, 5, 12])  # of 4, 20 and 48 rows: leaves of both kinds
@pytest.mark.parametrize("signs", [(1, -1), (-1, -2), (2, 1)])
@pytest.mark.parametrize("heavy", [700, 1100])
def test_scores_of_any_size(n, signs, heavy):
    """Scores of 1e34 and their like, of either sign, in the common pages and in a path's own: the largest takes all the weight."""
    u = torch.randn(256, generator=torch.Generator().manual_seed(4)).sign()
    k = (signs[1] * 1e14 * u).expand(1, 1, 1300, 256).clone()
    k[0, 0, heavy] = signs[0] * 1e14 * u
    k, v, v2 = k.bfloat16(), rows(2, 1, 1, 1000), rows(3, 5, 1, 300)
    c, o = forked(k[:, :, :1000], v, k[:, :, 1000:].expand(5, -1, -1, -1), v2)
    out = shared(c, (1e18 * u).expand(5, 4, n, 256).bfloat16().cuda(), causal=False, out_dtype=torch.float32)
    for s in range(5):
        want = o.values(s)[1][0, heavy]  # held exactly: one key, one weight
        assert np.allclose(f64(out[s]), want, rtol=2.0**-8, atol=0)
    assert c.device_status() == 0


@pytest.mark.parametrize("n", [1, 5, 12])
def test_masked_rows_cannot_leak(n):
    k, v, k2, v2 = rows(1, 1, 1, 1000), rows(2, 1, 1, 1000), rows(3, 5, 1, 200), rows(4, 5, 1, 200)
    for x, y in ((k, v), (k2, v2)):
        x[:, :, 4: x.shape[2] - 70], y[:, :, 4: x.shape[2] - 70] = -3e20, 3e20
    k2[:, :, :130], v2[:, :, :130] = rows(5, 5, 1, 130), rows(6, 5, 1, 130)
    c, o = forked(k, v, k2, v2)
    check(c, o, rows(9, 5, 4, n), window=120, sinks=4)


@pytest.mark.parametrize("n", [1, 5, 12])
def test_value_pages_of_very_different_sizes(n):
    v, v2 = rows(2, 1, 1, 960), rows(4, 5, 1, 320)
    sizes = [1, 1e-9, 1e6, 1e3, 1e-3, 0, 1e9, 1e-12, 1, 1e4]
    for x in (v, v2):
        for j in range(x.shape[2] // 64):
            x[:, :, 64 * j: 64 * j + 64] *= sizes[(j + x.shape[0]) % 10]
    c, o = forked(rows(1, 1, 1, 960) * 4, v, rows(3, 5, 1, 320) * 4, v2)
    check(c, o, rows(9, 5, 8, n))


@pytest.mark.parametrize("n", [1, 5, 12])
@pytest.mark.parametrize("sign", [1, -1])
def test_rising_scores_move_the_reference(n, sign):
    u = torch.randn(256, generator=torch.Generator().manual_seed(4))
    k = rows(1, 1, 1, 1500, dtype=torch.float32) * 0.2 + sign * u * torch.linspace(-6, 6, 1500)[None, None, :, None]
    k = k.bfloat16()
    c, o = forked(k[:, :, :1000], rows(2, 1, 1, 1000), k[:, :, 1000:].expand(6, -1, -1, -1), rows(3, 6, 1, 500))
    q = (u + 0.1 * rows(9, 6, 4, n).float()).bfloat16()
    check(c, o, q)
    check(c, o, q, causal=False)


@pytest.mark.parametrize("qs,ks,vs", [(1e-20, 1, 1), (1, 1e-9, 1e-9), (1e4, 1e-4, 1e10), (30, 1, 1), (1e15, 1e-15, 1e-20), (0, 1, 1), (1, 0, 1)])
@pytest.mark.parametrize("n", [1, 12])
def test_ranges(qs, ks, vs, n):
    c, o = forked(rows(1, 1, 1, 700) * ks, rows(2, 1, 1, 700) * vs, rows(3, 5, 1, 200) * ks, rows(4, 5, 1, 200) * vs)
    check(c, o, rows(9, 5, 4, n) * qs)
