"""The paged 8-bit cache on the GPU against its oracle: values held bit for bit,
page ids, sharing, and attention within bounds that follow from its roundings."""
import numpy as np
import pytest
import torch

from oracle import paged

pytestmark = pytest.mark.gpu


def rows(seed, E, H, n, outliers=False, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(E, H, n, 256, generator=g)
    if outliers:
        at = torch.rand(E, H, 1, 256, generator=g).topk(8, dim=-1).indices.expand(-1, -1, n, -1)
        x.scatter_(-1, at, 20 * x.gather(-1, at))
    return x.to(dtype)


def f64(t):
    return t.double().cpu().numpy()


def pair(slots, H, pages, max_tokens=None):
    """A device cache whose pool starts as NaN codes and scales, and its oracle."""
    from rotated_bit_quantized_gb300 import IQPagedCache
    c = IQPagedCache(slots, H, pages, max_tokens)
    c.k_codes.fill_(0x7F), c.v_codes.fill_(0xFF), c.k_scales.fill_(float("nan")), c.v_scales.fill_(float("nan")), c.table.fill_(-1)
    return c, paged.OraclePaged(slots, H, pages, c.max_pages)


def same(c, o):
    """Lengths, page ids, holders, the device's table and every value held."""
    assert c.lens.tolist() == o.lens and c._refs.tolist() == o.refs and c.pages_free == o.refs.count(0)
    table = c.table.cpu().numpy()
    for s in range(o.slots):
        assert c.page_ids(s).tolist() == o.rows[s]
        assert table[s, : len(o.rows[s])].tolist() == o.rows[s]
    n = max(o.lens) + 3
    k, v = c.read(0, n)
    k, v = f64(k), f64(v)
    for s in range(o.slots):
        ok, ov, _ = o.values(s)
        for got, want in ((k[s], ok), (v[s], ov)):
            assert (got[:, : o.lens[s]] == want).all()
            assert (got[:, o.lens[s]:] == 0).all()


def put(c, o, k, v, slots=None, counts=None):
    c.append(k.cuda(), v.cuda(), slots=slots, counts=counts)
    o.append(f64(k), f64(v), slots, counts)


def bounds(res, out_f32):
    """How far a result may be off: every weight p 2^e is held in two e4m3 parts (half a step twice: 2^-8 of it),
    cut from its fp16 form (half a step: 2^-11); a query element in two parts too (exact, but 2^-17 of the row's
    largest at the least code); sums of 256 products in fp32 (2^-16 of the sum of magnitudes); exp and the rest 2^-13.
    At the least codes a weight is off by half a step, and by half a step for the place where it is cut: 2^-9 in all,
    and the row's largest weight is at 2^5 or above then, so 2^-14 of that one."""
    out, weight, floor, slack = res
    tol = (2.0**-8 + 2.0**-11 + 2 * (2.0**-17 + 2.0**-16) * slack + 2.0**-13) * weight + 2.0**-14 * floor + 1e-30
    return tol if out_f32 else tol + 2.0**-8 * (np.abs(out) + tol)


def check_attend(c, o, q, out_dtype=torch.float32, slots=None, counts=None, scale=1 / 16, **kw):
    out = c.attend(q.cuda(), scale=scale, slots=slots, counts=counts, out_dtype=out_dtype, **kw)
    assert out.dtype == out_dtype and out.shape == q.shape
    res = paged.attend(o, f64(q), scale, slots, counts, **kw)
    got = f64(out)
    live = ~np.isnan(res[0])
    tol = bounds(res, out_dtype == torch.float32)
    d = np.abs(got - res[0])
    assert np.isfinite(got).all()
    assert (d[live] <= tol[live]).all(), (d[live] / tol[live]).max()
    if counts is not None:
        assert (got[~live] == 0).all()
    # Roundings of weights are random: their rms is well below their bound.  That does not go for a score's own
    # error, which moves a whole row: a fp32 sum of 256 products is off by up to 256 * 2^-24 = 2^-16 of the sum of
    # magnitudes (slack), the query's parts by 2^-17 of it, and exp makes of that twice as much of every p / sum p.
    # (Scores of 1e8, as in one case of test_ranges, are off by 6 from 2^-24 alone: any key near the top may win.)
    score = np.linalg.norm((2 * (2.0**-17 + 2.0**-16) * res[3] * res[1])[live])
    assert np.linalg.norm(d[live]) <= 2.0**-8 * np.linalg.norm(res[0][live]) + score + 1e-30
    assert c.device_status() == 0
    return got


# ------------------------------------------------------------------ values held

@pytest.mark.parametrize("H,steps", [(1, [1]), (2, [63, 1, 1]), (2, [64, 64]), (3, [1, 1, 1, 200, 5]), (1, [700, 1]), (8, [65, 3])])
@pytest.mark.parametrize("outliers", [False, True])
def test_appended_rows_bit_for_bit(H, steps, outliers):
    c, o = pair(3, H, 60, 800)
    for i, n in enumerate(steps):
        put(c, o, rows(10 + i, 3, H, n, outliers) * (1 + 3 * i), rows(30 + i, 3, H, n) / (1 + i), None, None)
        same(c, o)
    assert c.device_status() == 0


def test_ragged_counts_and_slot_lists():
    c, o = pair(6, 2, 80, 900)
    put(c, o, rows(1, 4, 2, 300, True), rows(2, 4, 2, 300), [5, 0, 3, 2], [300, 0, 1, 129])
    same(c, o)
    put(c, o, rows(3, 3, 2, 70), rows(4, 3, 2, 70), range(3, 6), np.array([70, 64, 63]))
    same(c, o)
    put(c, o, rows(5, 1, 2, 7), rows(6, 1, 2, 7), [0])
    same(c, o)


def test_strided_inputs():
    c, o = pair(2, 2, 10)
    k = rows(1, 2, 50, 2).transpose(1, 2)  # [entries, rows, heads, D] seen as [entries, heads, rows, D]
    v = rows(2, 4, 2, 50)[::2]
    assert not k.is_contiguous() and not v.is_contiguous()
    kc, vc = rows(1, 2, 50, 2).cuda().transpose(1, 2), rows(2, 4, 2, 50).cuda()[::2]
    c.append(kc, vc)
    o.append(f64(k), f64(v))
    same(c, o)


@pytest.mark.parametrize("big", [1e-38, 1e-13, 1e-6, 1.0, 448.0, 449.0, 1e10, 5e20, 3e38])
def test_magnitudes(big):
    c, o = pair(1, 1, 3)
    k = (rows(1, 1, 1, 20).float() * big).clamp(-3e38, 3e38).bfloat16()
    put(c, o, k, rows(2, 1, 1, 20))
    put(c, o, rows(3, 1, 1, 5), k[:, :, :5] * 0.5)
    same(c, o)
    over = (k.float().abs().max() > 448 * 2.0**60).item()
    assert bool(c.device_status() & 0x40000) == over
    assert c.device_status() == 0  # read once, cleared


def test_non_finite_values_are_held_finite():
    c, o = pair(1, 2, 3)
    k, v = rows(1, 1, 2, 30), rows(2, 1, 2, 30)
    k[0, 0, 3, 5], k[0, 1, 4, 6], v[0, 0, 29, 255] = float("nan"), float("inf"), float("-inf")
    put(c, o, k, v)
    same(c, o)
    assert c.device_status() & 0x40000
    assert not ((c.k_codes[0] & 0x7F) == 0x7F).any() and not ((c.v_codes[0] & 0x7F) == 0x7F).any()


def test_page_operations_against_the_oracle():
    rng = np.random.default_rng(5)
    c, o = pair(6, 2, 40, 700)
    done = {k: 0 for k in ("append", "full", "trim", "fork", "free", "compact")}
    for step in range(60):
        what = rng.integers(6)
        slots = [int(s) for s in rng.permutation(6)[: rng.integers(1, 4)]]
        if what <= 1:
            n = int(rng.choice([1, 2, 64, 130]))
            counts = [int(x) for x in rng.integers(0, n + 1, len(slots))]
            k, v = rows(100 + step, len(slots), 2, n, True), rows(200 + step, len(slots), 2, n)
            need = sum(-(-(o.lens[s] + m) // 64) - -(-o.lens[s] // 64) + bool(m and o.lens[s] % 64 and o.refs[o.rows[s][-1]] > 1)
                       for s, m in zip(slots, counts))
            if need > o.refs.count(0) or any(o.lens[s] + m > 704 for s, m in zip(slots, counts)):
                with pytest.raises(Exception, match="CAPACITY"):
                    c.append(k.cuda(), v.cuda(), slots=slots, counts=counts)
                done["full"] += 1
            else:
                put(c, o, k, v, slots, counts)
                done["append"] += 1
        elif what == 2:
            n = [int(x) for x in rng.integers(0, 90, len(slots))]
            assert c.trim(n, slots).tolist() == o.trim(n, slots)
            done["trim"] += 1
        elif what == 3:
            src = [int(s) for s in rng.integers(0, 6, len(slots))]
            c.fork(src, slots)
            o.fork(src, slots)
            done["fork"] += 1
        elif what == 4 and step % 3 == 0:
            c.free(slots)
            o.free(slots)
            done["free"] += 1
        elif what == 5:
            to = c.compact()
            assert to.pages == max(1, c.pages_used) and to.pages_free == to.pages - c.pages_used
            same(to, o.compact(to.pages))
            done["compact"] += 1
        same(c, o)
    assert all(done[k] for k in done if k != "full"), done
    assert c.device_status() == 0


def test_permuting_slots_is_one_call():
    c, o = pair(5, 1, 30)
    put(c, o, rows(1, 5, 1, 100), rows(2, 5, 1, 100), None, [100, 64, 10, 0, 65])
    c.fork([1, 2, 0, 4, 3], [0, 1, 2, 3, 4])
    o.fork([1, 2, 0, 4, 3], [0, 1, 2, 3, 4])
    same(c, o)
    c.fork([0, 0, 0], [0, 3, 1])  # one slot onto itself
    o.fork([0, 0, 0], [0, 3, 1])
    same(c, o)


def test_every_holder_of_a_page_goes_on_at_once():
    c, o = pair(4, 2, 12)
    put(c, o, rows(1, 1, 2, 70, True), rows(2, 1, 2, 70), [0])
    c.fork([0, 0, 0], [1, 2, 3])
    o.fork([0, 0, 0], [1, 2, 3])
    put(c, o, rows(3, 4, 2, 3) * 50, rows(4, 4, 2, 3) * 50)  # exponents grow in every copy
    same(c, o)
    assert c.pages_used == 5  # one shared full page, four last pages: the shared one was let go


def test_compact_into_a_given_cache_and_back():
    from rotated_bit_quantized_gb300 import IQPagedCache
    c, o = pair(4, 2, 40)
    put(c, o, rows(1, 4, 2, 300), rows(2, 4, 2, 300), None, [300, 1, 0, 257])
    c.fork([0], [2]), o.fork([0], [2])
    c.free([0]), o.free([0])
    snap, _ = pair(4, 2, 25)
    snap.append(rows(9, 4, 2, 80).cuda(), rows(8, 4, 2, 80).cuda())  # contents that are dropped
    assert c.compact(out=snap) is snap
    same(snap, o.compact(25))
    put(c, o, rows(5, 4, 2, 9), rows(6, 4, 2, 9))  # the snapshot does not follow
    back = o.compact(25)
    put(snap, back, rows(5, 4, 2, 9), rows(6, 4, 2, 9))
    with pytest.raises(Exception, match="CAPACITY"):
        c.compact(out=IQPagedCache(4, 2, 3))
    with pytest.raises(Exception, match="INVALID"):
        c.compact(out=c)
    # many short runs: every second page of a long slot
    c, o = pair(2, 1, 1500)
    for i in range(700):
        put(c, o, rows(i, 2, 1, 64), rows(i + 1, 2, 1, 64))
    c.free([0]), o.free([0])
    same(c.compact(), o.compact(700))


def fragmented():
    """Slot 2 and its fork 3 share a partly full page, slot 4 has one of its own, and the free pages lie one by one
    between slot 0's: a long append takes more runs of pages than one launch describes (256)."""
    c, o = pair(6, 1, 700, 320 * 64)
    for i in range(300):
        put(c, o, rows(i, 2, 1, 64), rows(i + 1, 2, 1, 64), [0, 1])
    put(c, o, rows(400, 2, 1, 70), rows(401, 2, 1, 70), [2, 4])
    c.fork([2], [3]), o.fork([2], [3])
    c.free([1]), o.free([1])
    k, v = rows(402, 3, 1, 150 * 64) * 40, rows(403, 3, 1, 150 * 64) * 40  # the exponents grow
    return c, o, k, v, dict(slots=[3, 4, 5], counts=[140 * 64 + 5, 3, 150 * 64 - 1])


def test_an_append_of_many_runs():
    c, o, k, v, kw = fragmented()
    put(c, o, k, v, **kw)
    same(c, o)
    put(c, o, k[:, :, :9], v[:, :, :9], slots=[2, 4, 5])  # the shared page went on in a copy
    same(c, o)


@pytest.mark.parametrize("launch", [0, 1])
def test_a_compaction_that_fails_at_a_launch(launch):
    """Into a cache that holds something: what it held, or, once its pages have been written over, nothing."""
    from rotated_bit_quantized_gb300 import IQError
    c, o, *_ = fragmented()
    put(c, o, rows(9, 1, 1, 200 * 64), rows(8, 1, 1, 200 * 64), [5])  # 300 runs of one page, and 200 more
    to, held = pair(6, 1, 700, 320 * 64)
    put(to, held, rows(1, 2, 1, 500), rows(2, 2, 1, 500), [1, 4])
    c._lib.iq_paged_debug_fail(launch)
    with pytest.raises(IQError, match="CUDA"):
        c.compact(out=to)
    same(c, o)
    same(to, held if launch == 0 else paged.OraclePaged(6, 1, 700, 320))
    assert c.compact(out=to) is to
    same(to, o.compact(700))


@pytest.mark.parametrize("launch", [0, 1])
def test_an_append_that_fails_at_a_launch_leaves_what_was_held(launch):
    from rotated_bit_quantized_gb300 import IQError
    c, o, k, v, kw = fragmented()
    c._lib.iq_paged_debug_fail(launch)  # on the host: that launch is not made
    with pytest.raises(IQError, match="CUDA"):
        c.append(k.cuda(), v.cuda(), **kw)
    same(c, o)
    put(c, o, k[:, :, :200], v[:, :, :200], [0, 1, 5])  # the pages it had taken go to others
    same(c, o)
    put(c, o, k, v, [3, 4, 1], kw["counts"])
    same(c, o)


# ------------------------------------------------------------------ attention

LENS = [[1], [64, 1, 65, 63, 2], [128, 127, 129, 0], [300, 0, 1025], [2000]]


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("Hq,H", [(1, 1), (16, 2), (6, 2), (5, 1), (8, 8), (64, 1)])
def test_decode(lens, Hq, H):
    c, o = pair(len(lens), H, 60)
    put(c, o, rows(1, len(lens), H, max(lens), True), rows(2, len(lens), H, max(lens)), None, lens)
    q = rows(3, len(lens), Hq, 1)
    check_attend(c, o, q)
    check_attend(c, o, q, torch.bfloat16, causal=False)


@pytest.mark.parametrize("lens", LENS[1:])
@pytest.mark.parametrize("Hq,H,n", [(16, 2, 4), (8, 1, 7), (3, 1, 5), (12, 4, 11), (8, 1, 16), (2, 2, 70), (12, 2, 33)])
def test_verify_and_chunks(lens, Hq, H, n):
    c, o = pair(len(lens), H, 60)
    put(c, o, rows(1, len(lens), H, max(lens), True), rows(2, len(lens), H, max(lens)), None, lens)
    q = rows(3, len(lens), Hq, n)  # some queries stand before the first token: zeros
    check_attend(c, o, q)
    check_attend(c, o, q, torch.bfloat16)
    check_attend(c, o, q, causal=False)


@pytest.mark.parametrize("n,length", [(129, 129), (200, 731), (513, 513)])
@pytest.mark.parametrize("Hq,H", [(8, 1), (6, 2), (3, 3)])
def test_prompts(n, length, Hq, H):
    c, o = pair(2, H, 40)
    put(c, o, rows(1, 2, H, length, True), rows(2, 2, H, length), None, [length, length - 70])
    q = rows(3, 2, Hq, n)
    check_attend(c, o, q)
    check_attend(c, o, q, counts=[n, n - 41])
    check_attend(c, o, q, causal=False)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (63, 0), (64, 1), (100, 64), (129, 70), (257, 4), (2**31 - 1, 0), (5, 2**31 - 1), (128, 128)])
@pytest.mark.parametrize("n", [1, 4, 150])
def test_windows_and_sinks(window, sinks, n):
    lens = [700, 3, 0, 131, 1500, 64]
    c, o = pair(6, 2, 60)
    put(c, o, rows(1, 6, 2, 1500, True), rows(2, 6, 2, 1500), None, lens)
    q = rows(3, 6, 8, n)
    check_attend(c, o, q, window=window, sinks=sinks)


def test_a_window_over_everything_is_causal_attention():
    c, o = pair(2, 2, 40)
    put(c, o, rows(1, 2, 2, 900), rows(2, 2, 2, 900))
    for n in (1, 5, 200):
        q = rows(3, 2, 16, n).cuda()
        assert torch.equal(c.attend(q), c.attend(q, window=900 + 5, sinks=0))


@pytest.mark.parametrize("n", [1, 3, 40])
def test_the_largest_window_and_sinks(n):
    """Also for queries before the first token, whose positions are negative."""
    c, o = pair(3, 2, 30, 500)
    put(c, o, rows(1, 3, 2, 450), rows(2, 3, 2, 450), None, [450, 2, 129])
    q = rows(3, 3, 8, n)
    for kw in (dict(window=2**31 - 1), dict(window=2**31 - 1, sinks=2**31 - 1), dict(window=449, sinks=2**31 - 1), dict(window=450)):
        assert (check_attend(c, o, q, **kw) == check_attend(c, o, q)).all()


@pytest.mark.parametrize("n", [1, 3, 40])
@pytest.mark.parametrize("scale", [-0.3, 0.0, 1e-30])
def test_scales_that_turn_or_level_the_scores(n, scale):
    c, o = pair(2, 2, 30, 500)
    put(c, o, rows(1, 2, 2, 450), rows(2, 2, 2, 450), None, [450, 131])
    check_attend(c, o, rows(3, 2, 8, n), scale=scale)


def test_counts_and_slots():
    c, o = pair(7, 2, 60)
    put(c, o, rows(1, 7, 2, 400, True), rows(2, 7, 2, 400), None, [400, 1, 64, 0, 333, 128, 200])
    for n, counts in [(1, [1, 0, 1, 1]), (6, [6, 3, 0, 1]), (140, [140, 77, 0, 1])]:
        for slots in ([6, 0, 3, 4], [4, 4, 1, 4]):
            q = rows(3, 4, 16, n)
            check_attend(c, o, q, slots=slots, counts=counts)
            out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
            got = c.attend(q.cuda(), slots=slots, counts=counts, out=out)
            assert got is out
            for i, m in enumerate(counts):
                assert (out[i, :, m:] == 7.0).all()  # rows that do not exist are left as they were
                assert not (out[i, :, :m] == 7.0).all() or m == 0


@pytest.mark.parametrize("n", [1, 9, 130])
def test_masked_rows_cannot_leak(n):
    """Rows outside every query's sight hold huge values: no trace of them in what is seen."""
    c, o = pair(1, 1, 12)
    k, v = rows(1, 1, 1, 600), rows(2, 1, 1, 600)
    v[0, 0, 4:300] = 3e20
    k[0, 0, 4:300] = -3e20
    put(c, o, k, v)
    c.trim(20), o.trim([20])  # stale rows behind the length
    q = rows(3, 1, 8, n)
    check_attend(c, o, q, window=100, sinks=4)
    check_attend(c, o, q[:, :, :1], window=250, sinks=0)


@pytest.mark.parametrize("n", [1, 4, 140])
def test_a_bad_query_spoils_its_own_rows_only(n):
    c, o = pair(2, 2, 12)
    put(c, o, rows(1, 2, 2, 300), rows(2, 2, 2, 300))
    q = rows(3, 2, 8, n).cuda()
    good = c.attend(q)
    bad = q.clone()
    bad[0, 3, n // 2, 7] = float("nan")
    bad[1, 0, 0, 9] = float("inf")
    got = c.attend(bad)
    spoilt = torch.zeros(2, 8, n, dtype=torch.bool, device="cuda")
    spoilt[0, 3, n // 2] = spoilt[1, 0, 0] = True
    assert torch.isnan(got[spoilt]).all()
    assert torch.equal(got[~spoilt], good[~spoilt])


@pytest.mark.parametrize("qs,ks,vs", [(1e-30, 1, 1), (1e4, 1e-4, 1e-6), (30, 1, 1e5), (1e18, 1e-10, 1e15), (0, 1, 1), (1, 0, 1e-9)])
@pytest.mark.parametrize("n", [1, 130])
def test_ranges(qs, ks, vs, n):
    c, o = pair(1, 1, 12)
    put(c, o, rows(1, 1, 1, 500) * ks, rows(2, 1, 1, 500) * vs)
    check_attend(c, o, rows(3, 1, 4, n) * qs)


@pytest.mark.parametrize("n", [1, 4, 130])
@pytest.mark.parametrize("signs", [(1, -1), (-1, -2), (2, 1)])
def test_scores_of_any_size(n, signs):
    """Scores of 1e34 and their like, of either sign: the largest takes all the weight, also over several ranges of keys."""
    c, o = pair(1, 1, 60)
    u = torch.randn(256, generator=torch.Generator().manual_seed(4)).sign()
    k = (signs[1] * 1e14 * u).expand(1, 1, 3000, 256).clone()
    k[0, 0, 1234] = signs[0] * 1e14 * u
    v = rows(2, 1, 1, 3000)
    put(c, o, k.bfloat16(), v)
    q = (1e18 * u).expand(1, 4, n, 256).bfloat16()
    out = c.attend(q.cuda(), causal=False, out_dtype=torch.float32)
    want = o.values(0)[1][0, 1234]  # held exactly: one key, one weight
    assert np.allclose(f64(out), want, rtol=2.0**-8, atol=0) and c.device_status() == 0


@pytest.mark.parametrize("n", [1, 130])
def test_value_pages_of_very_different_sizes(n):
    c, o = pair(1, 1, 12)
    v = rows(2, 1, 1, 640)
    for j in range(10):
        v[:, :, 64 * j: 64 * j + 64] *= [1, 1e-9, 1e6, 1e3, 1e-3, 0, 1e9, 1e-12, 1, 1e4][j]
    put(c, o, rows(1, 1, 1, 640) * 4, v)
    check_attend(c, o, rows(3, 1, 8, n))


@pytest.mark.parametrize("n", [1, 140])
def test_rising_scores_move_the_reference(n):
    """Keys in order of their scores, and in the opposite order: the running maximum moves at every step, or never."""
    for sign in (1, -1):
        c, o = pair(1, 1, 30)
        k = rows(1, 1, 1, 1500, dtype=torch.float32) * 0.2
        u = torch.randn(256, generator=torch.Generator().manual_seed(4))
        k += sign * u * torch.linspace(-6, 6, 1500)[None, None, :, None]
        put(c, o, k.bfloat16(), rows(2, 1, 1, 1500))
        q = (u + 0.1 * rows(3, 1, 4, n).float()).bfloat16()
        check_attend(c, o, q)
        check_attend(c, o, q, causal=False)


@pytest.mark.parametrize("n", [1, 4, 140])
@pytest.mark.parametrize("spread", [0.0, 0.05, 1.0])
def test_one_heavy_key_and_a_long_flat_tail(n, spread):
    """Half of the weight on the first key, half on 16384 others, whose values have a common part: each small weight
    lies near or below e4m3's least codes, but what they lose must not add up.  2^-8 and 2^-11 for the parts of the
    heavy key.  The tail: 64 weights of a page are cut at 64 evenly spaced places of a step of 2^-9, so their sum is
    off by half a step at most where they are equal: 2^-16 each, 16384 of them, against a sum of 2 * 2^5: 2^-8.
    Not equal ones are off by 2^-9 / sqrt(3) each at random: 128 * 2^-9.8 / 2^6 = 2^-8.8; the bound takes three of it."""
    N = 16384
    c, o = pair(1, 1, 260)
    g = torch.Generator().manual_seed(7)
    u = torch.randn(256, generator=g).sign() * 0.25  # |u|^2 = 16
    k = torch.zeros(1, 1, N + 1, 256)
    k[0, 0, 1:] = torch.randn(N, 1, generator=g) * spread * u
    k[0, 0, 0] = 8 * u  # score 8 * 16 * scale
    k, v = k.bfloat16(), (1 + 0.25 * torch.randn(1, 1, N + 1, 256, generator=g)).bfloat16()
    v[0, 0, 0] *= -1  # the two halves nearly cancel: an error of either shows
    put(c, o, k, v)
    q = (u * (1 + 0 * torch.arange(4 * n).view(1, 4, n, 1))).bfloat16()
    scale = np.log(N) / 128  # the heavy key's weight is that of all others together
    out, weight = paged.attend(o, f64(q), scale, causal=False)[:2]
    got = f64(c.attend(q.cuda(), scale=scale, causal=False, out_dtype=torch.float32))
    assert (np.abs(got - out) <= (2.0**-8 + 2.0**-11 + 3 * 2.0**-8.8 + 2.0**-13) * weight).all()


@pytest.mark.parametrize("n", [1, 4, 8, 12, 24, 140])
@pytest.mark.parametrize("N", [4096, 32768, 131072])
@pytest.mark.parametrize("spread", [0.0, 1.0])
def test_small_weights_beside_a_heavy_key(n, N, spread):
    """Half of the weight on one key whose value is 0, as on a first token that only draws attention: what comes out is
    what N small weights leave, on values without a common part.  Every weight is held in two e4m3 parts to 2^-8 of it
    (and 2^-11 for its fp16 form), and, where it lies below 2^-8 of the largest among its 32 keys, to 2^-9 or worse of
    what then hardly counts; the errors go with the values' signs, so the result is off by as much, in norm, at most;
    then exp and the scores' own error (slack, see check_attend), which moves all small weights alike."""
    H = 2
    c, o = pair(1, 1, N // 64 + 2)
    g = torch.Generator().manual_seed(N + n)
    u = torch.randn(256, generator=g).sign() * 0.25  # |u|^2 = 16
    k = torch.randn(1, 1, N + 1, 1, generator=g) * spread / np.log(N) * 8 * u
    k[0, 0, 777] = 8 * u
    v = torch.randn(1, 1, N + 1, 256, generator=g)
    v[0, 0, 777] = 0
    put(c, o, k.bfloat16(), v.bfloat16())
    q = u.expand(1, H, n, 256).bfloat16()
    scale = np.log(N) / 128
    out, weight, floor, slack = paged.attend(o, f64(q), scale, causal=False)
    got = f64(c.attend(q.cuda(), scale=scale, causal=False, out_dtype=torch.float32))
    off = np.linalg.norm(got - out) / np.linalg.norm(out)
    assert off <= 2.0**-8 + 2.0**-9 + 2.0**-11 + 2.0**-13 + 2 * (2.0**-17 + 2.0**-16) * slack.max(), off


@pytest.mark.parametrize("n", [1, 4, 8, 24])
def test_a_key_that_dominates_gives_its_values(n):
    """The last of 3001 keys weighs 1 - 2^-10.  Its weight enters numerator and sum as it is held, so its rounding
    cancels: what is left is 2^-8 of the others' share, twice, and the fp32 score's error times that share."""
    c, o = pair(1, 1, 60)
    g = torch.Generator().manual_seed(11)
    u = torch.randn(256, generator=g).sign() * 0.25
    k = torch.randn(1, 1, 3001, 1, generator=g) * 0.01 * u
    k[0, 0, 3000] = 7.3 * u
    put(c, o, k.bfloat16(), rows(2, 1, 1, 3001))
    q = u.expand(1, 2, n, 256).bfloat16()
    scale = np.log(3000 * 2.0**10) / (7.3 * 16)
    out, weight, _, slack = paged.attend(o, f64(q), scale, causal=False)
    got = f64(c.attend(q.cuda(), scale=scale, causal=False, out_dtype=torch.float32))
    largest = np.abs(o.values(0)[1]).max()
    share = 2.0**-9  # of the others, and their effect on the sum
    assert (np.abs(got - out) <= share * (2 * 2.0**-8 + 2.0**-13 + 2 * (2.0**-17 + 2.0**-16) * slack) * largest + 2.0**-22 * np.abs(out)).all()


def test_append_attend_is_both_calls():
    for lens, n, nq in [([100, 0, 64, 63], 1, 1), ([500, 3, 1, 0], 4, 4), ([130, 700, 0, 64], 150, 150), ([70, 5, 9, 200], 3, 1)]:
        a, o = pair(5, 2, 60)
        put(a, o, rows(1, 4, 2, 700), rows(2, 4, 2, 700), [4, 1, 2, 0], lens)
        a.fork([4], [3]), o.fork([4], [3])
        b = a.compact(out=pair(5, 2, 60)[0])
        k, v, q = rows(3, 4, 2, n).cuda(), rows(4, 4, 2, n).cuda(), rows(5, 4, 16, nq).cuda()
        kw = dict(slots=[3, 0, 1, 4])
        if n == nq and n > 1:
            kw["counts"] = [n, n - 1, 1, n]
        got = a.append_attend(k, v, q, **kw)
        b.append(k, v, **kw)
        assert torch.equal(got, b.attend(q, **kw))
        o.append(f64(k), f64(v), **kw)
        same(a, o)


def test_results_do_not_change_from_call_to_call():
    c, o = pair(3, 2, 200)
    put(c, o, rows(1, 3, 2, 4000), rows(2, 3, 2, 4000), None, [4000, 77, 1300])
    for n in (1, 4, 300):
        q = rows(3, 3, 16, n).cuda()
        want = c.attend(q)
        for _ in range(5):
            assert torch.equal(c.attend(q), want)


# ------------------------------------------------------------------ streams, graphs, places

def test_calls_on_two_streams_at_once():
    c, o = pair(2, 2, 300)
    put(c, o, rows(1, 2, 2, 8000), rows(2, 2, 2, 8000))
    qs = [rows(3 + i, 2, 16, n).cuda() for i, n in enumerate((1, 4, 1, 200))]
    want = [c.attend(q) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    for _ in range(5):
        got = []
        for s, q in zip(streams, qs):
            with torch.cuda.stream(s):
                got.append(c.attend(q))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_host_threads_on_one_stream():
    import threading
    c, o = pair(2, 2, 300)
    put(c, o, rows(1, 2, 2, 8000), rows(2, 2, 2, 8000))
    qs = [rows(3 + i, 2, 16, n).cuda() for i, n in enumerate((1, 4, 1, 200))]
    want = [c.attend(q) for q in qs]
    torch.cuda.synchronize()
    got = [[] for _ in qs]

    def work(i):
        for _ in range(30):
            got[i].append(c.attend(qs[i]))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(qs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert all(len(g) == 30 and all(torch.equal(x, w) for x in g) for g, w in zip(got, want))


def test_captured_calls_replay_with_their_lengths():
    c, o = pair(3, 2, 60)
    put(c, o, rows(1, 2, 2, 500), rows(2, 2, 2, 500), [0, 1], [500, 130])
    k, v, q = rows(3, 2, 2, 1).cuda(), rows(4, 2, 2, 1).cuda(), rows(5, 2, 16, 1).cuda()
    big = rows(6, 2, 16, 140).cuda()
    c.attend(big), c.attend(q)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step = c.append_attend(k, v, q)
            wide = c.attend(big)
        graphs.append((g, step, wide))
        if len(graphs) == 1:
            o.append(f64(k), f64(v))
    # the first graph appends row 500 / 130, the second row 501 / 131; inputs are read at replay
    k2, v2, q2 = rows(7, 2, 2, 1), rows(8, 2, 2, 1), rows(9, 2, 16, 1)
    graphs[0][0].replay()
    torch.cuda.synchronize()
    res = paged.attend(o, f64(q), 1 / 16)
    assert (np.abs(f64(graphs[0][1]) - res[0]) <= bounds(res, False)).all()
    k.copy_(k2), v.copy_(v2), q.copy_(q2)
    graphs[1][0].replay()
    torch.cuda.synchronize()
    o.append(f64(k2), f64(v2))
    res = paged.attend(o, f64(q2), 1 / 16)
    assert (np.abs(f64(graphs[1][1]) - res[0]) <= bounds(res, False)).all()
    res = paged.attend(o, f64(big), 1 / 16)
    assert (np.abs(f64(graphs[1][2]) - res[0]) <= bounds(res, False)).all()
    same(c, o)
    # two graphs at once, each with a workspace of its own
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    gs = []
    for x in (q, big):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = c.attend(x)
        gs.append((g, y, c.attend(x)))
    torch.cuda.synchronize()
    for _ in range(5):
        for (g, _, _), s in zip(gs, (a, b)):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for _, y, want in gs)


def test_a_pool_past_32_bits():
    """A slot whose pages lie beyond 4 GB of codes."""
    from rotated_bit_quantized_gb300 import IQPagedCache
    low, H = 40000, 8  # 40000 pages * 8 heads * 16 KB = 5.2 GB of keys
    c, o = IQPagedCache(2, H, low + 40, 2000), paged.OraclePaged(2, H, 40, 32)
    c._refs[:low], c._desc.free_pages, c._desc.first_free = 1, 40, 0
    k, v = rows(1, 2, H, 700, True), rows(2, 2, H, 700)
    put(c, o, k, v)
    assert c.page_ids(0)[0] == low
    put(c, o, k[:, :, :1], v[:, :, :1])
    for n in (1, 130):
        check_attend(c, o, rows(3, 2, 2 * H, n))
    got = f64(c.read(0, 701)[1])
    assert (got[1] == o.values(1)[1]).all()
    c._refs[:low] = 0
    c._desc.free_pages += low
    c.free([1])
    c.fork([0], [1])
    assert (f64(c.compact().read(0, 701)[1])[1] == o.values(0)[1]).all()


@pytest.mark.parametrize("n", [1, 130])
def test_a_bad_page_id_sets_a_status_bit(n):
    """The device's table, written over by someone else: ids are kept inside the pool, and the status word tells."""
    c, o = pair(1, 1, 8)
    put(c, o, rows(1, 1, 1, 300), rows(2, 1, 1, 300))
    good = c.table.clone()
    for bad in (-1, 8, 2**31 - 1, -2**31):
        c.table[0, 2] = bad
        out = c.attend(rows(3, 1, 8, n).cuda())
        c.read(0, 300)
        assert torch.isfinite(out).all()
        assert c.device_status() == 0x80000
    c.table.copy_(good)
    check_attend(c, o, rows(3, 1, 8, n))


@pytest.mark.parametrize("Hq,n", [(4, 1), (16, 1), (16, 4), (16, 140)])
def test_waits_that_run_out_are_told(Hq, n):
    """No page is loaded, through a hook on the host: every wait for one ends after a second, the call returns, the
    status word tells, and the calls behind it are right."""
    c, o = pair(3, 2, 60)
    put(c, o, rows(1, 3, 2, 900), rows(2, 3, 2, 900), None, [900, 1, 129])
    q = rows(3, 3, Hq, n)
    check_attend(c, o, q)
    c._lib.iq_paged_debug_stall()
    c.attend(q.cuda())
    status = c.device_status()  # (of the roles that wait, each tells or sees that another one has given up)
    assert status & 0xB and not status & ~0xB
    check_attend(c, o, q)
    same(c, o)


def test_python_refusals():
    c, _ = pair(2, 2, 4)
    k, q = rows(1, 2, 2, 3).cuda(), rows(2, 2, 4, 3).cuda()
    for bad in (k.float(), k.cpu(), k[..., :128], k[0], k[:, :1]):
        with pytest.raises(ValueError):
            c.append(bad, bad)
    with pytest.raises(ValueError):
        c.append(k, k[:, :, :2])
    with pytest.raises(ValueError):
        c.append(k, k, slots=[0])
    with pytest.raises(ValueError):
        c.append(k, k, counts=[1.5, 1])
    with pytest.raises(ValueError):
        c.append(rows(1, 3, 2, 3).cuda(), rows(1, 3, 2, 3).cuda())
    for bad in (q.half(), q.cpu(), q[0]):
        with pytest.raises(ValueError):
            c.attend(bad)
    for out in (torch.empty(2, 4, 2, 256, device="cuda"), torch.empty(2, 4, 3, 256, device="cuda", dtype=torch.half),
                torch.empty(2, 4, 256, 3, device="cuda").transpose(2, 3), torch.empty(2, 4, 3, 256)):
        with pytest.raises(ValueError):
            c.attend(q, out=out)
    with pytest.raises(ValueError):
        c.attend(q, out=torch.empty(q.shape, device="cuda"), out_dtype=torch.bfloat16)
    for kw in (dict(window=-1), dict(sinks=3), dict(causal=False, window=3), dict(slots=[0, 2]), dict(counts=[4, 0]), dict(scale=float("inf"))):
        with pytest.raises(Exception, match="INVALID"):
            c.attend(q, **kw)
    with pytest.raises(Exception, match="UNSUPPORTED"):
        c.attend(rows(1, 2, 3, 1).cuda())
    assert c.lens.tolist() == [0, 0] and c.pages_free == 4 and c.device_status() == 0
    empty = c.attend(q)
    assert (empty == 0).all()  # empty slots: nothing is seen
    assert c.attend(q[:, :, :0]).shape == (2, 4, 0, 256)
    assert c.attend(q[:0]).shape == (0, 4, 3, 256)
    c.append(k[:, :, :0], k[:, :, :0])
    c.append(k[:0], k[:0])
    assert c.read(0, 0)[0].shape == (2, 2, 0, 256)
