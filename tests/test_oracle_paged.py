"""Pins of the paged 8-bit cache's oracle: the e4m3 rounding against the table of
all codes, the page exponent, the page model against a list of rows, and the
attention against a second, key-by-key way."""
import numpy as np
import pytest

from oracle import paged


def codes():
    """Every finite e4m3 value from its bits: sign, 4 exponent bits (bias 7), 3 fraction bits."""
    out = []
    for b in range(256):
        e, f = b >> 3 & 15, b & 7
        if e == 15 and f == 7:
            continue  # NaN
        v = f / 8 * 2.0**-6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        out.append(-v if b >> 7 else v)
    return np.array(sorted(set(out)))


def test_e4m3_is_the_nearest_code_with_ties_to_even():
    table = codes()
    assert len(table) == 2 * 127 - 1 and table.max() == 448.0
    rng = np.random.default_rng(0)
    y = np.concatenate([table, (table[1:] + table[:-1]) / 2, rng.standard_normal(4000) * np.exp2(rng.uniform(-12, 9, 4000))])
    got = paged.e4m3(y)
    near = np.abs(table[None] - y[:, None])
    assert np.isin(got, table).all()
    assert (np.abs(got - y) <= near.min(1)).all()
    for v, g in zip(y, got):  # ties: the even fraction
        d = np.abs(table - v)
        if (d == d.min()).sum() == 2:
            a = abs(g)
            size = np.floor(np.log2(max(a, 2.0**-6)))
            assert a / 2.0 ** (size - 3) % 2 == 0
    assert paged.e4m3(1e9) == 448.0 and paged.e4m3(-500.0) == -448.0


@pytest.mark.parametrize("top,e", [(0.0, -40), (448.0, 0), (448.0001, 1), (224.0, -1), (1.75, -8), (1.7500001, -7), (1.0, -8),
                                   (2.0**-60, -40), (448.0 * 2.0**60, 60), (1e38, 60)])
def test_page_exponent(top, e):
    assert paged.page_exponent(top) == e


def test_error_bound_and_growth():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((1, 2, 40, 256))
    c = paged.OraclePaged(1, 2, 4)
    c.append(x[:, :, :10], x[:, :, :10])
    big = x[:, :, 10:] * 100  # grows the exponent: what was there is rounded again
    c.append(big, big)
    k, v, e = c.values(0)
    want = np.concatenate([x[0, :, :10], big[0]], 1)
    unit = np.exp2(e)[..., None]
    # half a step: 2^-4 of the value, or 2^-10 of the page's unit, twice for the rows rounded twice
    bound = np.maximum(2.0**-4 * np.abs(want), 2.0**-10 * unit) * np.where(np.arange(40) < 10, 2.2, 1.0)[None, :, None]
    assert (np.abs(k - want) <= bound).all() and (np.abs(v - want) <= bound).all()


def test_pages_against_a_list_of_rows():
    """Append, trim, fork, free and compact against lists of row numbers (rows held exactly: small powers of two)."""
    rng = np.random.default_rng(2)
    c = paged.OraclePaged(5, 1, 60)
    model = [[] for _ in range(5)]
    number = 0

    def rows(count):
        nonlocal number
        x = np.zeros((1, 1, count, 256))
        for j in range(count):
            number += 1
            x[0, 0, j, :16] = [number >> b & 1 for b in range(16)]  # the row's number in bits
            x[0, 0, j, 16] = 1.0
        return x, list(range(number - count + 1, number + 1))

    for _ in range(200):
        what, s = rng.integers(5), int(rng.integers(5))
        if what <= 1 and c.refs.count(0) > 6:
            x, ids = rows(int(rng.integers(1, 150)))
            c.append(x, x, [s])
            model[s] += ids
        elif what == 2:
            n = int(rng.integers(0, 100))
            assert c.trim(n, [s]) == [min(n, len(model[s]))]
            model[s] = model[s][: max(0, len(model[s]) - n)]
        elif what == 3:
            src, dst = [int(t) for t in rng.integers(0, 5, 2)], [int(t) for t in rng.permutation(5)[:2]]
            c.fork(src, dst)
            was = [list(m) for m in model]
            for a, b in zip(src, dst):
                model[b] = list(was[a])
        else:
            c.free([s])
            model[s] = []
        for cc in (c, c.compact()):
            used = set()
            for t in range(5):
                k, v, _ = cc.values(t)
                got = (k[0, :, :16] @ 2.0 ** np.arange(16)).astype(int).tolist()
                assert got == model[t] and (k == v).all()
                assert len(cc.rows[t]) == -(-len(model[t]) // 64)
                used |= set(cc.rows[t])
            assert {p for p, r in enumerate(cc.refs) if r} == used == set(cc.held)
        assert sorted(used) == list(range(len(used)))  # the compacted one's ids


@pytest.mark.parametrize("causal,window,sinks", [(True, 0, 0), (False, 0, 0), (True, 7, 0), (True, 3, 2), (True, 1, 5), (True, 200, 3)])
def test_attention_against_key_by_key(causal, window, sinks):
    rng = np.random.default_rng(3)
    lens = [0, 1, 5, 70]
    c = paged.OraclePaged(4, 2, 10)
    x = rng.standard_normal((2, 4, 2, 70, 256))
    c.append(x[0], x[1], counts=lens)
    q = rng.standard_normal((4, 6, 4, 256))
    out = paged.attend(c, q, 0.1, causal=causal, window=window, sinks=sinks)[0]
    for i, n in enumerate(lens):
        k, v, _ = c.values(i)
        for h in range(6):
            for j in range(4):
                p = n - 4 + j
                num, den = np.zeros(256), 0.0
                for t in range(n):
                    if causal and t > p or window and t <= p - window and t >= sinks:
                        continue
                    w = np.exp(0.1 * q[i, h, j] @ k[h // 3, t])
                    num, den = num + w * v[h // 3, t], den + w
                assert np.allclose(out[i, h, j], num / den if den else 0.0, rtol=1e-12, atol=1e-14)
