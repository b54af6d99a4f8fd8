"""Rotary positions on the GPU against the oracle in 64 bits: rows to rows, and into the pages of the 8-bit cache."""
import numpy as np
import pytest
import torch

from oracle import paged, rotary
from test_gpu_paged import f64, pair, rows

pytestmark = pytest.mark.gpu

U = 2.0**-24  # half a step of float32 at 1


def plan(rd=64, interleaved=False, norm=True, scaling="none", seed=9, **kw):
    """A plan and what the oracle needs of it."""
    from rotated_bit_quantized_gb300 import IQRotary
    g = torch.Generator().manual_seed(seed)
    w = [0.3 * torch.randn(256, generator=g) for _ in range(2)] if norm else [None, None]
    kw = dict(scaling=scaling, factor=8.0, original=4096) | kw
    rot = IQRotary(rd, interleaved=interleaved, q_norm=w[0], k_norm=w[1], eps=1e-6, norm_offset=1.0, **kw)
    lo, hi = {"yarn": (1, 32), "banded": (1, 4)}.get(scaling, (0, 0))
    f = [rotary.frequency(i, rd, 10000.0, scaling, 8.0, 4096, lo, hi) for i in range(rd // 2)]
    return rot, (w, f, interleaved, rot.amplitude)


def exact(x, at, ref, which):
    """x [entries, heads, n, 256] (a tensor) at positions [entries, n], in 64 bits, and a bound of its fp32 form's error:
    the sum of 256 squares (chains of 8, then 5 levels of a tree: 13 roundings, halved by the root), the root, two products:
    10 U of a normed element at most.  A cosine or sine: 2 units of the last place and the amplitude's product, below 8 U of
    the amplitude; a product and a sum: 2 U more.  The frequency's own 2^-53 and
    its turns' 2^-53, both relative, times the angle's size."""
    w, f, interleaved, amplitude = ref
    x = f64(x)
    if w[which] is not None:
        x = rotary.norm(x, 1.0 + w[which].double().numpy(), 1e-6)
    y = rotary.turn(x, at[:, None, :], f, interleaved, amplitude)
    n = len(f)
    size = np.abs(x)
    if n:
        a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
        both = (size[..., a] + size[..., b]) * amplitude
        size[..., a] = size[..., b] = both
    return y, size * (20 * U + 2.0**-51 * (1 + np.abs(at).max()))


def check(out, y, tol):
    got = f64(out)
    if out.dtype == torch.bfloat16:
        tol = tol + 2.0**-8 * (np.abs(y) + tol)
    assert (np.abs(got - y) <= tol).all(), (np.abs(got - y) / tol).max()


@pytest.mark.parametrize("rd,interleaved", [(0, False), (16, False), (64, False), (96, False), (128, False), (144, False), (192, False), (240, False), (256, False),
                                            (16, True), (80, True), (128, True), (144, True), (256, True)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("norm", [False, True])
def test_layouts(rd, interleaved, dtype, norm):
    rot, ref = plan(rd, interleaved, norm)
    q, k = rows(1, 3, 5, 37, True, dtype).cuda(), rows(2, 3, 2, 37, True, dtype).cuda()
    start = [0, 1000, 77]
    a, b = rot.apply(q, k, positions=start)
    assert a.shape == q.shape and b.shape == k.shape and a.dtype == dtype and a.is_contiguous()
    at = np.array(start)[:, None] + np.arange(37)
    check(a, *exact(q, at, ref, 0))
    check(b, *exact(k, at, ref, 1))


@pytest.mark.parametrize("E,H,n", [(1, 1, 1), (1, 17, 1), (7, 3, 1), (32, 16, 1), (256, 1, 1), (2, 40, 3), (1, 1, 513), (3, 18, 97), (2, 2, 2049)])
def test_sizes(E, H, n):
    rot, ref = plan()
    q = rows(3, E, H, n).cuda()
    out = rot.apply(q, positions=5)
    check(out, *exact(q, np.broadcast_to(5 + np.arange(n), (E, n)), ref, 0))


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn", "banded"])
def test_far_positions_and_scalings(scaling):
    rot, ref = plan(128, True, False, scaling)
    q = rows(4, 6, 2, 20, dtype=torch.float32).cuda()
    start = [0, 1 << 20, 10**6 + 7, (1 << 31) - 20, -5, -(1 << 31)]
    out = rot.apply(q, positions=start)
    at = np.array(start, dtype=np.int64)[:, None] + np.arange(20)
    check(out, *exact(q, at, ref, 0))


def test_positions_of_every_row():
    rot, ref = plan(96)
    q, k = rows(5, 4, 6, 50).cuda(), rows(6, 4, 2, 50).cuda()
    at = torch.randint(-100, 1 << 30, (4, 50), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    a, b = rot.apply(q, k, positions=at.cuda())
    check(a, *exact(q, at.numpy().astype(np.int64), ref, 0))
    check(b, *exact(k, at.numpy().astype(np.int64), ref, 1))
    c = rot.apply(q, positions=at.cuda().t().contiguous().t())  # strided positions
    assert torch.equal(a, c)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_views_of_a_projection(dtype):
    rot, ref = plan(256)
    x = rows(7, 1, 2, 33 * 8, dtype=dtype).view(2, 33, 8, 256).cuda()  # [entries, rows, heads, 256]
    q, k, v = x.transpose(1, 2).split([4, 2, 2], 1)
    a, b = rot.apply(q, k, positions=3)
    c, d = rot.apply(q.contiguous(), k.contiguous(), positions=3)
    assert torch.equal(a, c) and torch.equal(b, d)
    check(a, *exact(q, np.broadcast_to(3 + np.arange(33), (2, 33)), ref, 0))
    # rows that no kernel can read where they lie (an odd offset, dims apart): copied
    flat = torch.zeros(2 * 4 * 33 * 256 + 3, dtype=dtype, device="cuda")
    odd = flat[3:].view(2, 4, 33, 256)
    odd.copy_(q)
    assert torch.equal(rot.apply(odd, positions=3), a)
    assert torch.equal(rot.apply(q.transpose(2, 3).contiguous().transpose(2, 3), positions=3), a)
    # the same rows for every entry and head
    one = q[:1, :1].expand(3, 5, -1, -1)
    assert torch.equal(rot.apply(one, positions=3), a[:1, :1].expand(3, 5, -1, -1))


def test_extreme_rows():
    rot, (w, f, il, amp) = plan(32)
    x = torch.zeros(1, 1, 6, 256, dtype=torch.float32)
    x[0, 0, 1] = 1e30                      # squares beyond fp32
    x[0, 0, 2] = 1e-25                     # squares of nothing next to eps
    x[0, 0, 3, 5] = float("nan")
    x[0, 0, 4, 200] = float("inf")
    x[0, 0, 5] = 3e38
    out = f64(rot.apply(x.cuda()))
    assert (out[0, 0, 0] == 0).all() and np.isnan(out[0, 0, 3]).all()
    for r in (1, 2, 5):
        y, tol = exact(x[:, :, r:r + 1], np.array([[r]]), (w, f, il, amp), 0)
        assert (np.abs(out[0, 0, r] - y[0, 0, 0]) <= tol[0, 0, 0] + 1e-38).all()
    assert np.isnan(out[0, 0, 4, 200]) and (out[0, 0, 4, 32:200] == 0).all()
    for dtype in (torch.bfloat16, torch.float32):  # without a norm only the pairs of such elements are touched
        plain, _ = plan(32, norm=False)
        y = plain.apply(x.to(dtype).cuda())[0, 0]
        assert torch.isnan(y[3, 5]) and torch.isnan(y[3, 21]) and torch.isfinite(torch.cat([y[3, :5], y[3, 6:21], y[3, 22:]])).all()
        assert torch.isinf(y[4, 200]) and torch.isfinite(y[4, :200]).all()
        x[0, 0, 2, 20] = float("inf")  # one that turns: its pair's two, and no others
        y = plain.apply(x.to(dtype).cuda())[0, 0, 2]
        x[0, 0, 2, 20] = 1e-25
        assert (torch.isfinite(y) == torch.tensor([j not in (4, 20) for j in range(256)], device="cuda")).all()


def test_outputs_past_32_bits():
    """4.6 GB of results, from one row's strides of zero; and a cache's rows far apart in a large tensor."""
    rot, ref = plan(64)
    one = rows(1, 1, 1, 1).cuda()
    out = rot.apply(one.expand(3, 75, 20000, 256))
    want = rot.apply(one.expand(1, 1, 20000, 256))[0, 0]
    for e, h in ((0, 0), (1, 40), (2, 74)):
        assert torch.equal(out[e, h], want)
    del out
    from rotated_bit_quantized_gb300 import IQPagedCache
    x = torch.zeros(2, 2 * 10**9 // 2, dtype=torch.bfloat16, device="cuda")  # entries 2 GB apart
    q, k, v = rows(2, 2, 4, 70).cuda(), rows(3, 2, 2, 70).cuda(), rows(4, 2, 2, 70).cuda()
    views = []
    for at, t in ((0, q), (5 * 10**8, k), (9 * 10**8, v)):
        views.append(x[:, at:at + t[0].numel()].view(2, *t.shape[1:]))
        views[-1].copy_(t)
    a, b = IQPagedCache(2, 2, 8), IQPagedCache(2, 2, 8)
    assert torch.equal(a.append_rotary(*views, rot), b.append_rotary(q, k, v, rot))
    assert all(torch.equal(i, j) for i, j in zip(a.read(0, 70), b.read(0, 70)))


def test_many_heads():
    rot, ref = plan(128, True)
    q = rows(1, 1, 300, 9).cuda()
    check(rot.apply(q, q[:, :7], positions=4)[0], *exact(q, 4 + np.arange(9)[None], ref, 0))
    c, o = pair(1, 1, 4)
    check_append(c, o, rot, ref, rows(2, 1, 300, 70), rows(3, 1, 1, 70), rows(4, 1, 1, 70))


def test_nothing_to_turn_and_no_rows():
    rot, _ = plan(0, norm=False)
    q = rows(8, 2, 3, 9).cuda()
    assert torch.equal(rot.apply(q, positions=12), q)
    a, b = rot.apply(q[:, :, :0], q[:, :1, :0])
    assert a.shape == (2, 3, 0, 256) and b.shape == (2, 1, 0, 256)
    assert rot.apply(q[:0]).shape == (0, 3, 9, 256)


def test_refusals():
    from rotated_bit_quantized_gb300 import IQPagedCache
    rot, _ = plan()
    q = rows(1, 2, 4, 8).cuda()
    at = torch.zeros(2, 8, dtype=torch.int32, device="cuda")
    for args, kw in [((q.half(),), {}), ((q.cpu(),), {}), ((q[..., :128],), {}), ((q[0],), {}), ((q, q.float()), {}), ((q, q[:1]), {}), ((q, q[:, :, :7]), {}),
                     ((q,), dict(positions=1.5)), ((q,), dict(positions=[1, 2, 3])), ((q,), dict(positions=1 << 31)), ((q,), dict(positions=at[:1])),
                     ((q,), dict(positions=at.long())), ((q,), dict(positions=at.cpu())), ((q.expand(2, 4, 8, 256).repeat(129, 1, 1, 1),), {})]:
        with pytest.raises(ValueError):
            rot.apply(*args, **kw)
    c = IQPagedCache(4, 2, 10)
    k, v = rows(2, 2, 2, 8).cuda(), rows(3, 2, 2, 8).cuda()
    for args, kw in [((q, k.float(), v), {}), ((q, k, v[:, :1]), {}), ((q[:1], k, v), {}), ((q[:, :, :3], k, v), {}), ((q, k, v), dict(positions=at[:, :3])),
                     ((q, k, v), dict(slots=[0, 0])), ((q, k, v), dict(counts=[9, 1])), ((q, rows(2, 2, 3, 8).cuda(), rows(3, 2, 3, 8).cuda()), {})]:
        with pytest.raises((ValueError, RuntimeError)):
            c.append_rotary(*args[:3], rot, **kw)
    assert c.lens.tolist() == [0] * 4 and c.pages_free == 10


# ------------------------------------------------------------------ into pages

def check_append(c, o, rot, ref, q, k, v, slots=None, counts=None, positions=None):
    """Append to both; every key held is its page's code nearest to the exact one, or, where that lies as near to the
    border of two codes as fp32 can err, a neighbour; values and the pages' other rows are the oracle's."""
    E, H, n, _ = k.shape
    ids = list(range(E)) if slots is None else list(slots)
    cnt = [n] * E if counts is None else list(counts)
    before = [o.lens[s] for s in ids]
    at = np.array(before)[:, None] + np.arange(n) if positions is None else positions.numpy().astype(np.int64)
    y, tol = exact(k, at, ref, 1)
    junk = None if q is None else torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    del junk  # what the next allocation of that size finds
    out = c.append_rotary(None if q is None else q.cuda(), k.cuda(), v.cuda(), rot, slots=slots, counts=counts,
                          positions=None if positions is None else positions.cuda())
    o.append(y, f64(v), slots, counts)
    assert c.lens.tolist() == o.lens and c._refs.tolist() == o.refs
    table = c.table.cpu().numpy()
    kk, vv = (f64(t) for t in c.read(0, max(o.lens) + 1))
    scales = f64(c.k_scales)
    for i, s in enumerate(ids):
        assert table[s, : len(o.rows[s])].tolist() == o.rows[s]
        ok, ov, _ = o.values(s)
        assert (vv[s][:, : o.lens[s]] == ov).all() and (kk[s][:, o.lens[s]:] == 0).all()
        assert (kk[s][:, : before[i]] == ok[:, : before[i]]).all()
        new, want = kk[s][:, before[i]: o.lens[s]], y[i, :, : cnt[i]]
        unit = np.repeat(scales[o.rows[s]].T, 64, 1)[:, before[i]: o.lens[s], None]  # the pages' scales
        step = np.ldexp(unit, np.frexp(np.maximum(np.abs(want) / unit, 2.0**-6))[1] - 4)
        assert (np.abs(new - want) <= step / 2 + tol[i, :, : cnt[i]]).all()
        same = new == ok[:, before[i]:]
        assert (~same).sum() <= 0.001 * same.size  # (of a border's neighbourhood, 2^-18 of a step, 1e-5 is expected)
        for t in range(before[i], o.lens[s]):  # a neighbour stays one: the oracle goes on from the codes held
            for h in range(H):
                o.held[o.rows[s][t // 64]][0][h].codes[t % 64] = kk[s][h, t] / scales[o.rows[s][t // 64], h]
    if q is not None:
        yq, tq = exact(q, at, ref, 0)
        for i in range(E):
            check(out[i, :, : cnt[i]], yq[i, :, : cnt[i]], tq[i, :, : cnt[i]])
            assert (out[i, :, cnt[i]:] == 0).all()
    else:
        assert out is None
    return out


@pytest.mark.parametrize("rd,interleaved", [(0, False), (64, False), (160, False), (256, False), (64, True), (256, True)])
@pytest.mark.parametrize("norm", [False, True])
def test_append_layouts(rd, interleaved, norm):
    rot, ref = plan(rd, interleaved, norm)
    c, o = pair(3, 2, 40, 800)
    for i, n in enumerate((70, 1, 64, 133)):
        check_append(c, o, rot, ref, rows(i, 3, 6, n, True), rows(10 + i, 3, 2, n, True) * (1 + i), rows(20 + i, 3, 2, n) * (1 + i))
    assert c.device_status() == 0


@pytest.mark.parametrize("interleaved", [False, True])
def test_append_of_full_pages_at_every_dim(interleaved):
    """The table of a page's cosines is up to 64 KB of shared memory, 48 at 192 dims."""
    for rd in range(16, 257, 16):
        rot, ref = plan(rd, interleaved)
        for n in (62, 63, 130):
            c, o = pair(2, 1, 9)
            check_append(c, o, rot, ref, rows(1, 2, 1, n), rows(2, 2, 1, n), rows(3, 2, 1, n))
            assert c.device_status() == 0


@pytest.mark.parametrize("H,Hq", [(1, 1), (1, 8), (3, 33), (8, 8)])
def test_append_heads_and_padded_batches(H, Hq):
    rot, ref = plan(64)
    c, o = pair(5, H, 60, 900)
    check_append(c, o, rot, ref, rows(1, 4, Hq, 200), rows(2, 4, H, 200), rows(3, 4, H, 200), [4, 0, 1, 2], [200, 0, 1, 127])
    check_append(c, o, rot, ref, rows(4, 5, Hq, 1), rows(5, 5, H, 1), rows(6, 5, H, 1))
    check_append(c, o, rot, ref, None, rows(7, 2, H, 65), rows(8, 2, H, 65), [3, 2])
    at = torch.randint(0, 1 << 22, (2, 30), generator=torch.Generator().manual_seed(3), dtype=torch.int32)
    check_append(c, o, rot, ref, rows(9, 2, Hq, 30), rows(10, 2, H, 30), rows(11, 2, H, 30), [1, 0], [30, 7], positions=at)
    assert c.device_status() == 0


@pytest.mark.parametrize("rd,interleaved,norm,scaling", [(64, False, True, "none"), (256, False, True, "none"), (96, False, True, "yarn"), (160, False, False, "none"),
                                                         (128, True, True, "yarn"), (64, True, False, "none"), (128, False, True, "none"), (0, False, True, "none")])
def test_codes_are_the_nearest_to_the_exact_keys(rd, interleaved, norm, scaling):
    """Four million codes, of which fp32 alone would put some on the wrong side of a border; in fp64 a border is
    missed where a key lies within 2^-45 or so of it, once in 10^11."""
    from rotated_bit_quantized_gb300 import IQPagedCache, IQRotary
    E, H, n = 8, 2, 1024
    g = torch.Generator().manual_seed(5)
    w = (0.3 * torch.randn(256, generator=g) * 1024).round() / 1024 if norm else None  # 1 + w is exact
    rot = IQRotary(rd, interleaved=interleaved, scaling=scaling, factor=8.0, original=4096, k_norm=w, norm_offset=1.0)
    c = IQPagedCache(E, H, E * n // 64)
    k, v = rows(6, E, H, n, True).cuda(), rows(7, E, H, n).cuda()
    k[:, :, ::7] *= 0.01
    at = torch.randint(0, 1 << 17, (E, n), generator=g, dtype=torch.int32).cuda()
    at[0, :100] = 0
    c.append_rotary(None, k, v, rot, positions=at)
    y = k.double()
    if norm:
        y = y / (y.square().mean(-1, keepdim=True) + 1e-6).sqrt() * (1.0 + w.double().cuda())
    if rd:
        angle = (at.double()[..., None] * torch.from_numpy(rot.frequencies).cuda())[:, None]
        a, b = (y[..., :rd:2], y[..., 1:rd:2]) if interleaved else (y[..., : rd // 2], y[..., rd // 2: rd])
        x, z = rot.amplitude * (a * angle.cos() - b * angle.sin()), rot.amplitude * (a * angle.sin() + b * angle.cos())
        y = torch.cat([torch.stack([x, z], -1).flatten(-2) if interleaved else torch.cat([x, z], -1), y[..., rd:]], -1)
    scale = c.k_scales[c.table[:, : n // 64].long()].double().transpose(1, 2).repeat_interleave(64, 2)[..., None]
    z = y / scale
    step = torch.exp2(torch.floor(torch.log2(z.abs().clamp_min(2.0**-6))) - 3)
    held = c.read(0, n)[0].double() / scale
    assert (held == (torch.round(z / step) * step)).all()
    assert c.device_status() == 0


def test_append_copies_shared_pages():
    rot, ref = plan(64)
    c, o = pair(4, 2, 30, 400)
    check_append(c, o, rot, ref, None, rows(1, 1, 2, 100), rows(2, 1, 2, 100), [0])
    c.fork([0, 0, 0], [1, 2, 3])
    o.fork([0, 0, 0], [1, 2, 3])
    check_append(c, o, rot, ref, rows(3, 4, 4, 3), rows(4, 4, 2, 3) * 50, rows(5, 4, 2, 3) * 50, None, [3, 2, 0, 1])
    assert c.device_status() == 0


def test_append_of_what_is_not_finite():
    from rotated_bit_quantized_gb300 import _abi
    rot, _ = plan(64, norm=False)
    k, v = rows(1, 1, 2, 3), rows(2, 1, 2, 3)
    for bad, status in ((float("nan"), _abi.IQ_STATUS_RANGE), (float("inf"), _abi.IQ_STATUS_RANGE), (3e38, _abi.IQ_STATUS_RANGE), (1e20, 0)):
        for which in (0, 1):
            c, _ = pair(1, 2, 2)
            x = [k.clone(), v.clone()]
            x[which][0, 1, 1, 200] = bad
            c.append_rotary(None, x[0].cuda(), x[1].cuda(), rot)
            held = [f64(t) for t in c.read(0, 3)]
            assert all(np.isfinite(t).all() for t in held)
            assert c.device_status() == status
            if bad != bad:
                assert held[which][0, 1, 1, 200] == 0 and np.abs(held[which]).max() < 10
            elif status:
                assert held[which][0, 1, 1, 200] == 448.0 * 2.0**60


def test_a_large_append_equals_small_ones():
    """More pages and entries than one launch's list of runs holds, past 2^16 rows."""
    rot, _ = plan(128)
    from rotated_bit_quantized_gb300 import IQPagedCache
    a, b = IQPagedCache(3, 1, 3400), IQPagedCache(3, 1, 3400)
    a.append(*(rows(s, 3, 1, 64).cuda() for s in (1, 2)), counts=[64, 0, 64])
    a.free([0])  # pages no longer in a row
    b.append(*(rows(s, 3, 1, 64).cuda() for s in (1, 2)), counts=[0, 0, 64])
    q, k, v = (rows(5 + i, 2, h, 1, ).expand(2, h, 66000, 256) for i, h in enumerate((2, 1, 1)))
    x = [t.clone().cuda() for t in (q, k, v)]
    out = a.append_rotary(*x, rot, slots=[0, 1])
    parts = [b.append_rotary(*(t[:, :, i:i + 22000] for t in x), rot, slots=[0, 1]) for i in range(0, 66000, 22000)]
    assert torch.equal(out, torch.cat(parts, 2))
    for s in (0, 65000, 21990):
        assert all(torch.equal(i, j) for i, j in zip(a.read(s, 900, slots=[0, 1]), b.read(s, 900, slots=[0, 1])))
    assert a.device_status() == 0 and b.device_status() == 0


# ------------------------------------------------------------------ streams, graphs, chains

def test_replays_in_a_graph_on_another_stream():
    rot, _ = plan(64)
    from rotated_bit_quantized_gb300 import IQPagedCache
    q, k, v = rows(1, 4, 8, 1).cuda(), rows(2, 4, 2, 1).cuda(), rows(3, 4, 2, 1).cuda()
    a, b = IQPagedCache(4, 2, 16), IQPagedCache(4, 2, 16)
    for c in (a, b):
        c.append(*(rows(s, 4, 2, 100).cuda() for s in (4, 5)))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            turned = rot.apply(q, k, positions=100)
            out = a.append_rotary(q, k, v, rot)
            att = a.attend(out)
        for i in range(3):
            q.copy_(rows(50 + i, 4, 8, 1)), k.copy_(rows(60 + i, 4, 2, 1)), v.copy_(rows(70 + i, 4, 2, 1))
            g.replay()
    torch.cuda.current_stream().wait_stream(s)
    want = b.append_rotary(q, k, v, rot)
    x, y = rot.apply(q, k, positions=100)
    assert torch.equal(out, want) and torch.equal(turned[0], x) and torch.equal(turned[1], y)
    assert torch.equal(att, b.attend(want))
    assert a.device_status() == 0 and b.device_status() == 0


def test_a_plan_made_on_a_busy_stream_is_ready_for_others():
    x, (w, *_) = rows(1, 2, 4, 30).cuda(), plan(128)[1]
    want = plan(128)[0].apply(x, x, positions=7)
    w = [t.cuda() for t in w]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)  # some 10 ms
        from rotated_bit_quantized_gb300 import IQRotary
        rot = IQRotary(128, scaling="none", q_norm=w[0], k_norm=w[1], norm_offset=1.0)
    got = rot.apply(x, x, positions=7)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_chains_of_calls_without_waits():
    """Each call reads what the one before hands out; the rotated cache's attention reads its queries early."""
    from rotated_bit_quantized_gb300 import IQCache, IQPagedCache, Rotation
    rot, _ = plan(64)
    so4 = Rotation(0)
    q = rows(1, 8, 8, 1).cuda()
    k, v = rows(2, 8, 2, 1).cuda(), rows(3, 8, 2, 1).cuda()
    past = [rows(s, 8, 2, 2000).cuda() for s in (4, 5)]

    def chain(wait):
        c, p = IQCache(8, 2, capacity=2304), IQPagedCache(8, 2, 8 * 34)
        c.append(*past, so4)
        p.append(*past)
        x, res = q, []
        for i in range(6):
            a, b = rot.apply(x, k, positions=2000 + i)
            wait()
            x = c.append_attend(b, v, a, so4)
            wait()
            x = p.append_rotary(x, k, v, rot)
            wait()
            x = c.attend(x, so4)
            wait()
            x = p.attend(x)
            wait()
            res.append(x)
        return res
    want = chain(torch.cuda.synchronize)
    for _ in range(5):
        got = chain(lambda: None)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_float32_cache_takes_turned_rows():
    from rotated_bit_quantized_gb300 import IQCache, Rotation
    rot, ref = plan(128, True, scaling="yarn")
    so4 = Rotation(0)
    q, k, v = (rows(i, 2, h, 40, dtype=torch.float32).cuda() for i, h in ((1, 4), (2, 2), (3, 2)))
    a, b = rot.apply(q, k)
    c = IQCache(2, 2, k_bits=8, v_bits=8, dtype=torch.float32)
    c.append(b, v, so4)
    out = f64(c.attend(a[:, :, -1:].contiguous(), so4))
    at = np.broadcast_to(np.arange(40), (2, 40))
    yq, yk = exact(q, at, ref, 0)[0], exact(k, at, ref, 1)[0]
    s = np.einsum("ehd,ehtd->eht", yq[:, :, -1].reshape(2, 4, 256), np.repeat(yk, 2, 1)) / 16
    p = np.exp(s - s.max(-1, keepdims=True))
    want = np.einsum("eht,ehtd->ehd", p / p.sum(-1, keepdims=True), np.repeat(f64(v), 2, 1))
    # 8 bits of groups whose elements span some 8: half a step of 8 / 255 in a value; a score of 256 such products
    # of keys off by as much at random moves by 0.02 * |q| / 16, some 0.03 of the weights
    assert np.abs(out[:, :, 0] - want).max() < 0.1


def keys_at_a_border(want):
    """Pairs (a, b) of bf16 numbers, positions and a frequency whose first turned element is 448 but for 2^-26 of it, from 64 bits."""
    w, got = 0.7310585786300049, []
    p = np.arange(1, 40000, dtype=np.float64)[:, None]
    a = 256 + 2.0 * np.arange(128)
    c, s = np.cos(p * w), np.sin(p * w)
    b = torch.from_numpy((a * c - 448) / s).to(torch.bfloat16).double().numpy()
    y, z = a * c - b * s, a * s + b * c
    off = np.abs(y / 448 - 1)
    at = np.argwhere((off < 2.0**-26) & (off > 2.0**-40) & (np.abs(z) < 440))  # (angles in 64 bits are off by 2^-38 of this at most)
    for i, j in at[:want]:
        got.append((a[j], b[i, j], int(p[i, 0]), y[i, j]))
    return w, got


@pytest.mark.parametrize("interleaved", [False, True])
def test_page_exponents_are_those_of_the_exact_keys(interleaved):
    """The least e with the page's largest exact key at most 448 * 2^e: where float32 cannot tell, it is not asked."""
    from rotated_bit_quantized_gb300 import IQPagedCache, IQRotary
    w, found = keys_at_a_border(256)
    n = len(found)
    assert n >= 64 and {y > 448 for *_, y in found} == {True, False}
    for rd in (16, 64, 96, 256):
        rot = IQRotary(rd, interleaved=interleaved, frequencies=[w] * (rd // 2))
        c = IQPagedCache(n, 1, n)
        k = torch.zeros(n, 1, 3, 256)
        at = torch.zeros(n, 3, dtype=torch.int32)
        first, second = (4, 5) if interleaved else (2, 2 + rd // 2)
        for i, (a, b, p, _) in enumerate(found):
            r = i % 3
            k[i, 0, r, first], k[i, 0, r, second], at[i, r] = a, b, p
            k[i, 0, (r + 1) % 3, 200] = 7.0
        k = k.to(torch.bfloat16).cuda()
        c.append_rotary(None, k, torch.zeros_like(k), rot, positions=at.cuda())
        want = [2.0 if y > 448 else 1.0 for *_, y in found]
        assert c.k_scales[:, 0].tolist() == want
        assert c.device_status() == 0


def test_page_exponents_of_normed_keys():
    from rotated_bit_quantized_gb300 import IQPagedCache, IQRotary
    g = np.random.default_rng(1)
    seen = set()
    for i in range(40):
        x = torch.from_numpy(g.standard_normal(256)).to(torch.bfloat16)
        x[i] = 9.0
        unit = 9.0 / np.sqrt((x.double().numpy() ** 2).mean() + 1e-6)
        weight = np.float32(448.0 / unit)
        y = float(weight) * unit
        if abs(y / 448 - 1) < 2.0**-45:
            continue
        rot = IQRotary(64 if i % 2 else 0, k_norm=torch.full((256,), float(weight)))
        c = IQPagedCache(1, 1, 1)
        k = x.view(1, 1, 1, 256).cuda()
        c.append_rotary(None, k, k, rot)
        assert c.k_scales.item() == (2.0 if y > 448 else 1.0), i
        seen.add(y > 448)
    assert seen == {True, False}


@pytest.mark.parametrize("base", [1e4, 1e7])
def test_float32_sines_of_small_angles(base):
    """Each product of a result is off by a few roundings of its own, also where the angle is a small part of a turn: a
    cosine or sine by 2, its product by 1, their sum by 2 and its correction: 6 U, and 2 for the angle's own
    reduction (held to 2^-24 of it and to 2^-54 of a turn); the frequency's 2^-52 times the position besides."""
    from rotated_bit_quantized_gb300 import IQRotary
    rot = IQRotary(256, base=base)
    x = torch.zeros(4, 1, 300, 256)
    g = torch.Generator().manual_seed(1)
    x[0, :, :, 128:] = torch.randn(1, 300, 128, generator=g)
    x[1, :, :, :128] = torch.randn(1, 300, 128, generator=g)
    x[2, :, :, 128:], x[2, :, :, :128] = torch.randn(1, 300, 128, generator=g), 1e-6 * torch.randn(1, 300, 128, generator=g)
    x[3] = x[0]
    at = np.stack([np.arange(300), np.arange(300), np.arange(300), 100000 - np.arange(300)])
    out = f64(rot.apply(x.cuda(), positions=torch.from_numpy(at).int().cuda()))
    a, b = f64(x)[..., :128], f64(x)[..., 128:]
    angle = (at[..., None] * rot.frequencies)[:, None]
    c, s, slip = np.cos(angle), np.sin(angle), 2.0**-51 * angle + 2.0**-52
    for got, want, tol in ((out[..., :128], a * c - b * s, np.abs(a * c) + np.abs(b * s)), (out[..., 128:], a * s + b * c, np.abs(a * s) + np.abs(b * c))):
        assert (np.abs(got - want) <= 8 * U * tol + slip * (np.abs(a) + np.abs(b))).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_large_eps_beside_squares_past_32_bits(dtype):
    """Sums of squares that pass float32 still have eps added to their mean."""
    from rotated_bit_quantized_gb300 import IQRotary
    x = torch.full((1, 1, 3, 256), 2.0**60, dtype=dtype)
    x[0, 0, 1] = 2.0**62
    x[0, 0, 2] = 2.0**100
    for eps in (1e-6, 1e30, 1e37, 3e38):
        rot = IQRotary(0, q_norm=torch.ones(256), k_norm=torch.ones(256), eps=eps)
        y = f64(x) / np.sqrt((f64(x) ** 2).mean(-1, keepdims=True) + eps)
        check(rot.apply(x.cuda()), y, 10 * U * np.abs(y))


@pytest.mark.parametrize("rd,interleaved,norm", [(64, False, True), (128, True, False), (96, False, True)])
def test_codes_where_the_amplitude_is_rounded_to_float32(rd, interleaved, norm):
    """An amplitude as far from float32's numbers as it may be: the codes are the nearest to the keys of that one."""
    from rotated_bit_quantized_gb300 import IQPagedCache, IQRotary
    E, H, n = 8, 2, 1024
    g = torch.Generator().manual_seed(5)
    w = (0.3 * torch.randn(256, generator=g) * 1024).round() / 1024 if norm else None  # 1 + w is exact
    rot = IQRotary(rd, interleaved=interleaved, k_norm=w, norm_offset=1.0, amplitude=1 + 2.0**-23 * 3 + 2.0**-24 * 0.99)
    c = IQPagedCache(E, H, E * n // 64)
    k = rows(6, E, H, n, True).cuda()
    at = torch.randint(0, 1 << 17, (E, n), generator=g, dtype=torch.int32).cuda()
    c.append_rotary(None, k, k, rot, positions=at)
    y = k.double()
    if norm:
        y = y / (y.square().mean(-1, keepdim=True) + 1e-6).sqrt() * (1.0 + w.double().cuda())
    angle = (at.double()[..., None] * torch.from_numpy(rot.frequencies).cuda())[:, None]
    a, b = (y[..., :rd:2], y[..., 1:rd:2]) if interleaved else (y[..., : rd // 2], y[..., rd // 2: rd])
    x, z = rot.amplitude * (a * angle.cos() - b * angle.sin()), rot.amplitude * (a * angle.sin() + b * angle.cos())
    y = torch.cat([torch.stack([x, z], -1).flatten(-2) if interleaved else torch.cat([x, z], -1), y[..., rd:]], -1)
    scale = c.k_scales[c.table[:, : n // 64].long()].double().transpose(1, 2).repeat_interleave(64, 2)[..., None]
    z = y / scale
    step = torch.exp2(torch.floor(torch.log2(z.abs().clamp_min(2.0**-6))) - 3)
    held = c.read(0, n)[0].double() / scale
    assert (held == (torch.round(z / step) * step)).all()
    top = z.abs().unflatten(2, (-1, 64)).amax((-1, -2))
    assert (top <= 448).all() and (top > 224).all()  # the least exponent
    assert c.device_status() == 0
