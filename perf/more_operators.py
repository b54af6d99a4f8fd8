"""Operators around the paged 8-bit cache as a user's program calls them, and their plain forms.

The cache: pages of 64 tokens for all kv heads, head_dim 256, codes in e4m3 with one power-of-two scale per page and head
(keys and values apart), one row of page ids per sequence slot.

kind        one pass
"rotate"    queries and keys, as views of a projection's output: each head's vector normed (root mean square, a weight per dim),
            then its first `rotary` dims turned by the token's position
"append"    the same for the queries and keys of new rows, the keys and the projection's values quantised into the slots' pages;
            the rotated queries and the touched pages' rows, read back as the values held, are the result
"shared"    attention of the last `rows` positions of `groups` x `paths` slots: all share their first `common` tokens, the paths of a
            group `branch` tokens more, and each has tokens of its own (window > 0: only the last `window` positions and the first `sinks` tokens)
"""
import math

import numpy as np
import torch

own = False

PAGE, DIM, E_MIN, E_MAX, TOP, EPS, BASE = 64, 256, -40, 60, 448.0, 1e-6, 10000.0
FACTOR, ORIGINAL = 8.0, 16384  # of the scaled position rules: how far a context is stretched, and from which length


def listed():
    def rotate(name, entries, rows, **more):
        return {"name": name, "kind": "rotate", "entries": entries, "rows": rows, "q_heads": 16, "kv_heads": 2, "rotary": 64, "interleaved": False,
                "scaling": "none", "norm": True, "start": 20000, "ids": False, "dtype": "bfloat16"} | more

    def append(name, entries, rows, tokens, **more):
        return {"name": name, "kind": "append", "entries": entries, "rows": rows, "tokens": tokens, "spread": 0, "ragged": False, "q_heads": 16, "kv_heads": 2,
                "rotary": 64, "interleaved": False, "scaling": "none", "norm": True} | more

    def shared(name, groups, paths, common, branch, tail, **more):
        return {"name": name, "kind": "shared", "groups": groups, "paths": paths, "common": common, "branch": branch, "tail": tail, "spread": 0, "rows": 1,
                "q_heads": 16, "kv_heads": 2, "window": 0, "sinks": 0} | more

    return [
        # one generated token of 32 sequences: the smallest call, latency
        rotate("rotate_step", 32, 1),
        # a batch of prompt chunks
        rotate("rotate_prompts", 16, 2048),
        # a float32 cache's queries and keys far into a stretched context: neighbouring dims paired, the whole head turned, no norm
        rotate("rotate_far_f32", 1, 2047, q_heads=12, kv_heads=4, rotary=256, interleaved=True, scaling="yarn", norm=False, start=1000000, dtype="float32"),
        # a few ragged prompts whose tokens carry positions of their own, as many kv heads as query heads
        rotate("rotate_ids", 5, 777, q_heads=8, kv_heads=8, rotary=96, interleaved=True, scaling="linear", ids=True),
        # one generated token for each of 32 sequences at lengths of their own: the decode step's write
        append("append_step", 32, 1, 2000, spread=1500),
        # a batch of fresh prompts, the benchmark's append shape
        append("append_prompts", 32, 4096, 0),
        # a padded batch of chunks of odd sizes behind histories of odd lengths, the whole head turned
        append("append_ragged", 7, 513, 1000, spread=999, ragged=True, q_heads=8, kv_heads=4, rotary=256, scaling="banded", norm=False),
        # one prompt of a chat tried along four paths: the smallest call, latency
        shared("paths_chat", 1, 4, 1024, 0, 16),
        # a long prompt along 32 paths
        shared("paths_long", 1, 32, 32768, 0, 100, spread=90),
        # drafted trees: a common prompt, three branches of it, five paths of each, four tokens each; other head counts
        shared("tree_verify", 3, 5, 16384, 2001, 300, spread=290, rows=4, q_heads=12, kv_heads=4),
        # a server's batch: one system prompt, 128 conversations of their own
        shared("system_prompt", 1, 128, 8192, 0, 2048, spread=2000),
        # a long prompt along 24 paths under a window with sinks
        shared("paths_window", 1, 24, 20000, 0, 130, spread=100, window=4096, sinks=4),
    ]


def _between(rng, low, high):
    """An odd or even whole number, spread over its logarithm."""
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high + 0.5))))))


def draw(rng):
    kind = rng.choice(["rotate", "rotate", "append", "append", "shared", "shared", "shared"])
    kv_heads = rng.choice([1, 2, 4, 8])
    q_heads = kv_heads * rng.choice([1, 2, 3, 4, 6, 8])
    case = {"kind": kind, "q_heads": q_heads, "kv_heads": kv_heads}
    if kind == "shared":
        groups, paths = rng.choice([1, 1, 1, 2, 3, 5]), _between(rng, 2, 40)
        rows = rng.choice([1, 1, 1, 2, 3, 5])
        room = 900000 // kv_heads  # tokens times kv heads of all slots, as the plain form lays them out
        tail = _between(rng, rows, max(rows, min(3000, room // (4 * groups * paths))))
        common = _between(rng, 64, max(65, min(40000, room // (2 * groups * paths))))
        branch = rng.choice([0, _between(rng, 1, max(2, min(4000, room // (4 * groups * paths))))])
        window = rng.choice([0, 0, 0, _between(rng, 1, 6000)])
        return case | {"groups": groups, "paths": paths, "common": common, "branch": branch, "tail": tail, "spread": rng.randrange(0, tail - rows + 1), "rows": rows,
                       "window": window, "sinks": rng.choice([0, 1, 4, 70]) if window else 0}
    entries = _between(rng, 1, 48)
    rows = _between(rng, 1, max(1, 900000 // (entries * (q_heads + 2 * kv_heads))))
    case |= {"entries": entries, "rows": rows, "rotary": rng.choice([16, 32, 64, 96, 128, 192, 256]), "interleaved": rng.random() < 0.5,
             "scaling": rng.choice(["none", "none", "linear", "yarn", "banded"]), "norm": rng.random() < 0.6}
    if kind == "rotate":
        return case | {"start": _between(rng, 1, 2000000), "ids": rng.random() < 0.3, "dtype": rng.choice(["bfloat16", "bfloat16", "float32"])}
    tokens = rng.randrange(0, 3000)
    return case | {"tokens": tokens, "spread": tokens // 2, "ragged": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs

def _lens(tokens, spread, n):
    """n lengths: `tokens`, give or take `spread`, the same for every seed; the first the shortest."""
    return [tokens - spread + (2 * spread * ((7 * b) % n)) // max(1, n - 1) for b in range(n)]


def _counts(case):
    """How many of an entry's rows there are: all, or, in a padded batch, half of them and more."""
    rows = case["rows"]
    return [rows - ((5 * b) % case["entries"]) * (rows // 2) // case["entries"] if case["ragged"] else rows for b in range(case["entries"])]


def _rows(g, lead, heads, rows, kind):
    """bf16 rows [lead, heads, rows, 256]: standard normals; keys have eight channels per head twenty times as large."""
    x = torch.randn(lead, heads, rows, DIM, generator=g, device="cuda")
    if kind == "keys":
        at = torch.rand(lead, heads, 1, DIM, generator=g, device="cuda").topk(8, dim=-1).indices
        x.scatter_(-1, at.expand(-1, -1, rows, -1), 20.0 * x.gather(-1, at.expand(-1, -1, rows, -1)))
    return x.to(torch.bfloat16)


def _projected(g, case):
    """What a layer's projection hands over: [entries, rows, (query heads, kv heads, kv heads) x 256], a few channels of
    every head larger; and the norms' weights, held as their difference from 1."""
    e, n, heads = case["entries"], case["rows"], case["q_heads"] + 2 * case["kv_heads"]
    dtype = getattr(torch, case.get("dtype", "bfloat16"))
    x = torch.randn(e, n, heads * DIM, generator=g, device="cuda")
    x.mul_(torch.where(torch.rand(heads * DIM, generator=g, device="cuda") < 0.03, 8.0, 1.0))
    weights = [(0.2 * torch.randn(DIM, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2)] if case["norm"] else [None, None]
    return x.to(dtype), weights


def _ids(g, case):
    """Positions that tokens carry: every entry's run from its start, with some tokens at one place (an image's, a tree's)."""
    step = (torch.rand(case["entries"], case["rows"], generator=g, device="cuda") < 0.7).int()
    return (case["start"] + step.cumsum(1)).to(torch.int32)


def _pages(tokens):
    return (tokens + PAGE - 1) // PAGE


def _tails(case):
    return _lens(case["tail"], case["spread"], case["groups"] * case["paths"])


def _history(g, case):
    """Keys and values of a "shared" case: of the common prompt [1, ...], of the branches [groups, ...], of the paths' own tokens [slots, ...], padded."""
    heads, slots = case["kv_heads"], case["groups"] * case["paths"]
    return [[_rows(g, lead, heads, max(1, rows), w) for w in ("keys", "values")]
            for lead, rows in ((1, case["common"]), (case["groups"], case["branch"]), (slots, max(_tails(case))))]


def _plan(case):
    """The framework's rotary plan, kept by a program."""
    from rotated_bit_quantized_gb300 import IQRotary

    return lambda weights: IQRotary(case["rotary"], base=BASE, interleaved=case["interleaved"], scaling=case["scaling"], factor=FACTOR, original=ORIGINAL,
                                    q_norm=weights[0], k_norm=weights[1], eps=EPS, norm_offset=1.0)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kind = case["kind"]
    st = {"case": case}
    if kind == "shared":
        parts = _history(g, case)
        st["q"] = _rows(g, case["groups"] * case["paths"], case["q_heads"], case["rows"], "queries")
        if own:
            st["cache"] = _own_tree(case, parts)
        else:
            st["pool"] = _plain_tree(case, parts)
        return st
    if kind == "append":
        lens = _lens(case["tokens"], case["spread"], case["entries"])
        past = [_rows(g, case["entries"], case["kv_heads"], max(1, max(lens)), w) for w in ("keys", "values")]
        st |= {"lens": lens, "counts": _counts(case)}
        if own:
            from rotated_bit_quantized_gb300 import IQPagedCache

            room = [t + case["rows"] for t in lens]
            st["cache"] = IQPagedCache(case["entries"], case["kv_heads"], sum(map(_pages, room)), max_tokens=max(room))
            st["cache"].append(*past, counts=lens)
        else:
            width = max(_pages(t + case["rows"]) for t in lens)
            st["pool"] = [_plain_pages(x, [torch.tensor(lens, device="cuda")], width) for x in past]
    st["x"], weights = _projected(g, case)
    st["ids"] = _ids(g, case) if kind == "rotate" and case["ids"] else None
    # the plan that a program keeps: the framework's where own is true, the frequencies and the weights else
    if own:
        st["rotary"] = _plan(case)(weights)
    else:
        st["weights"] = weights
        st["freq"], st["amplitude"] = torch.from_numpy(_frequencies(case)).cuda(), _amplitude(case)
    return st


def _own_tree(case, parts):
    from rotated_bit_quantized_gb300 import IQPagedCache

    groups, paths = case["groups"], case["paths"]
    slots, tails = groups * paths, _tails(case)
    stem = case["common"] + case["branch"]
    pages = _pages(case["common"]) + groups * (1 + _pages(case["branch"])) + sum(1 + _pages(t) for t in tails)
    cache = IQPagedCache(slots, case["kv_heads"], pages, max_tokens=stem + max(tails))
    cache.append(*parts[0], slots=[0])
    leaders = range(0, slots, paths)
    if groups > 1:
        cache.fork([0] * (groups - 1), leaders[1:])
    if case["branch"]:
        cache.append(*parts[1], slots=leaders)
    others = [b for b in range(slots) if b % paths]
    cache.fork([b - b % paths for b in others], others)
    cache.append(*parts[2], slots=range(slots), counts=tails)
    return cache


# ------------------------------------------------------------------ one pass

def run(state):
    return _own(state) if own else _plain(state)


def _heads(st):
    """Queries, keys and values as views of the projection's output: [entries, heads, rows, 256]."""
    case = st["case"]
    q, k = case["q_heads"], case["kv_heads"]
    return st["x"].unflatten(-1, (q + 2 * k, DIM)).transpose(1, 2).split([q, k, k], dim=1)


def _own(st):
    case = st["case"]
    if case["kind"] == "shared":
        return st["cache"].attend(st["q"], window=case["window"], sinks=case["sinks"], shared=True)
    q, k, v = _heads(st)
    if case["kind"] == "rotate":
        return st["rotary"].apply(q, k, positions=case["start"] if st["ids"] is None else st["ids"])
    cache = st["cache"]
    cache.trim(cache.lens - st["lens"])
    q = cache.append_rotary(q, k, v, st["rotary"], counts=st["counts"] if case["ragged"] else None)
    keys, values = cache.read([t - t % PAGE for t in st["lens"]], case["rows"] + PAGE)
    return q, keys, values


def _plain(st):
    case = st["case"]
    if case["kind"] == "shared":
        return _plain_attend(st)
    q, k, v = _heads(st)
    dev = q.device
    if case["kind"] == "rotate":
        at = st["ids"] if st["ids"] is not None else (case["start"] + torch.arange(case["rows"], device=dev)).expand(case["entries"], -1)
        return tuple(_plain_rotary(st, x, at, w).to(x.dtype) for x, w in zip((q, k), st["weights"]))
    lens, counts = (torch.tensor(st[w], device=dev) for w in ("lens", "counts"))
    j = torch.arange(case["rows"], device=dev)
    at, live = lens[:, None] + j, j < counts[:, None]
    q = torch.where(live[:, None, :, None], _plain_rotary(st, q, at, st["weights"][0]), 0.0).to(torch.bfloat16)
    return q, _plain_append(st["pool"][0], _plain_rotary(st, k, at, st["weights"][1]), lens, counts), _plain_append(st["pool"][1], v.float(), lens, counts)


# ------------------------------------------------------------------ plain forms

def _frequencies(case):
    """The radians per position of every pair of turned dims, fp64."""
    n = case["rotary"] // 2
    f = BASE ** (-np.arange(n, dtype=np.float64) / n)
    slow = f / FACTOR
    if case["scaling"] == "linear":
        return slow
    if case["scaling"] == "yarn":  # pairs that turn over 32 times within the original length stay, under once are stretched
        pair = lambda turns: n * math.log(ORIGINAL / (turns * 2 * math.pi)) / math.log(BASE)  # noqa: E731
        low, high = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), 2 * n - 1)
        ramp = np.clip((np.arange(n) - low) / max(high - low, 0.001), 0, 1)
        return slow * ramp + f * (1 - ramp)
    if case["scaling"] == "banded":  # wavelengths below a quarter of the original length stay, above it are stretched, a blend between
        keep = np.clip((ORIGINAL * f / (2 * math.pi) - 1.0) / (4.0 - 1.0), 0, 1)
        return slow * (1 - keep) + f * keep
    return f


def _amplitude(case):
    return 0.1 * math.log(FACTOR) + 1.0 if case["scaling"] == "yarn" else 1.0


def _plain_rotary(st, x, at, weight):
    """x [entries, heads, rows, 256] normed and turned, fp32; the angles of far positions in fp64."""
    case = st["case"]
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * (1.0 + weight.float())
    angle = (at.double()[..., None] * st["freq"])[:, None]
    c, s = ((t * st["amplitude"]).float() for t in (angle.cos(), angle.sin()))
    turned, rest = x.split([case["rotary"], DIM - case["rotary"]], dim=-1)
    a, b = turned.unflatten(-1, (-1, 2)).unbind(-1) if case["interleaved"] else turned.chunk(2, dim=-1)
    both = a * c - b * s, a * s + b * c
    return torch.cat([torch.stack(both, -1).flatten(-2) if case["interleaved"] else torch.cat(both, -1), rest], -1)


def _exponent(top):
    """The least e with top <= 448 * 2^e, within its limits."""
    m, x = torch.frexp(top)  # top = m * 2^x, 0.5 <= m < 1;  448 = 0.875 * 2^9
    return torch.where(top > 0, x - 9 + (m > 0.875).int(), torch.full_like(x, E_MIN)).clamp(E_MIN, E_MAX)


def _power(e):
    """2^e in fp32, bit by bit: a power function need not be exact."""
    return ((e + 127) << 23).view(torch.float32)


def _codes(paged, e):
    return (paged / _power(e)[..., None, None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn)


def _add_rows(pool, x, begin, end):
    """Rows [begin, end) of x [lead, heads, width * 64, 256] join what the pages hold: codes [lead, heads, width, 64, 256], exponents."""
    t = torch.arange(x.shape[2], device=x.device)
    new = ((t >= begin[:, None]) & (t < end[:, None]))[:, None, :, None]
    fresh = torch.where(new, x.float(), 0.0).unflatten(2, (-1, PAGE))
    e = _exponent(fresh.abs().amax((-2, -1)))
    if pool is not None:
        e = torch.maximum(e, pool[1])
        fresh += pool[0].float() * _power(pool[1])[..., None, None]
    return _codes(fresh, e), e


def _plain_pages(x, ends, width):
    """Pages filled by one append for each of `ends` (rows [0, ends[0]), then [ends[0], ends[1]), ...) of x [lead, heads, rows, 256]."""
    x = torch.nn.functional.pad(x, (0, 0, 0, width * PAGE - x.shape[2]))
    pool, begin = None, torch.zeros_like(ends[0])
    for end in ends:
        pool, begin = _add_rows(pool, x, begin, end), end
    return pool


def _plain_append(pool, x, lens, counts):
    """The pages' rows from the one that each entry goes on in, as held after the append: bf16 [entries, heads, rows + 64, 256]."""
    lead, heads, n, _ = x.shape
    codes, exps = pool
    first, width = lens // PAGE, 1 + (n + PAGE - 1) // PAGE
    at = first[:, None] + torch.arange(width, device=x.device)
    inside = (at < codes.shape[2])[:, None, :]
    pick = at.clamp(max=codes.shape[2] - 1)
    here = torch.arange(lead, device=x.device)[:, None]
    held = torch.where(inside[..., None, None], codes.view(torch.uint8)[here, :, pick].transpose(1, 2), 0).view(torch.float8_e4m3fn)
    e = torch.where(inside, exps[here, :, pick].transpose(1, 2), E_MIN)
    place = (lens % PAGE)[:, None] + torch.arange(n, device=x.device)
    rows = torch.zeros(lead, heads, width * PAGE, DIM, device=x.device)
    rows.scatter_(2, place[:, None, :, None].expand(-1, heads, -1, DIM), x)
    codes, e = _add_rows((held, e), rows, lens % PAGE, lens % PAGE + counts)
    return (codes.float() * _power(e)[..., None, None]).flatten(2, 3)[:, :, : n + PAGE].to(torch.bfloat16)


def _whole(case, parts, w):
    """Every slot's own copy of its rows [slots, heads, tokens, 256] (w: 0 keys, 1 values), and where its three appends end."""
    slots, paths = case["groups"] * case["paths"], case["paths"]
    common, branch, tail = (p[w] for p in parts)
    x = torch.cat([common[:, :, : case["common"]].expand(slots, -1, -1, -1), branch[:, :, : case["branch"]].repeat_interleave(paths, 0), tail], 2)
    lens = torch.tensor(_tails(case), device=x.device) + case["common"] + case["branch"]
    return x, [torch.full_like(lens, case["common"]), torch.full_like(lens, case["common"] + case["branch"]), lens]


def _plain_tree(case, parts):
    pool = []
    for w in (0, 1):
        x, ends = _whole(case, parts, w)
        pool.append(_plain_pages(x, ends, _pages(x.shape[2])))
    return pool + [ends[-1]]


def _plain_attend(st):
    case, (keys, values, lens) = st["case"], st["pool"]
    lead, heads, rows = len(lens), case["kv_heads"], case["rows"]
    rep = case["q_heads"] // heads
    k, v = ((c.float() * _power(e)[..., None, None]).flatten(2, 3) for c, e in (keys, values))
    t = torch.arange(k.shape[2], device=k.device)
    at = (lens[:, None] - rows + torch.arange(rows, device=k.device))[:, :, None]
    see = t <= at
    if case["window"]:
        see &= (t > at - case["window"]) | (t < case["sinks"])
    s = (st["q"].float().reshape(lead, heads, rep * rows, DIM) @ k.transpose(-1, -2)).mul_(1.0 / math.sqrt(DIM)).unflatten(2, (rep, rows))
    s.masked_fill_(~see[:, None, None], -math.inf)
    p = s.sub_(s.amax(-1, keepdim=True)).exp_()
    out = (p.flatten(2, 3) @ v).unflatten(2, (rep, rows)) / p.sum(-1, keepdim=True)
    return out.reshape(lead, case["q_heads"], rows, DIM).to(torch.bfloat16)


# ------------------------------------------------------------------ work

def work(case):
    rows, q_heads, heads = case["rows"], case["q_heads"], case["kv_heads"]
    if case["kind"] == "rotate":
        moved = case["entries"] * rows * (q_heads + heads) * DIM
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": 2 * moved * size + (4 * case["entries"] * rows if case["ids"] else 0), "flops": 10 * moved}
    if case["kind"] == "append":
        n = sum(_counts(case))
        first = sum(t % PAGE for t in _lens(case["tokens"], case["spread"], case["entries"]))  # the rows that read-back finds in front
        turned, back = n * q_heads * 2 * 2 * DIM, (n + first) * 2 * heads * 3 * DIM  # bf16 in and out; codes in, bf16 out
        return {"bytes": turned + n * 2 * heads * 3 * DIM + back, "flops": 10 * n * (q_heads + 2 * heads) * DIM}
    common, stem = case["common"], case["common"] + case["branch"]
    slots, lens = case["groups"] * case["paths"], [stem + t for t in _tails(case)]
    pairs, low = 0, []  # low: the first key behind the sinks that a slot's rows see
    for t in lens:
        for at in range(t - rows, t):
            begin = max(0, at - case["window"] + 1) if case["window"] else 0
            pairs += at + 1 - begin + min(case["sinks"], begin)
        low.append(max(0, t - rows - case["window"] + 1) if case["window"] else 0)
    seen = lambda b, e, x: max(0, e - max(b, x)) + max(0, min(case["sinks"], x, e) - b)  # of keys [b, e): those from x on, and sinks  # noqa: E731
    paths = case["paths"]
    keys = seen(0, common, min(low)) + sum(seen(common, stem, min(low[i:i + paths])) for i in range(0, slots, paths)) + sum(seen(stem, t, x) for t, x in zip(lens, low))
    return {"bytes": slots * q_heads * rows * 2 * 2 * DIM + keys * heads * 2 * DIM, "flops": 4 * DIM * q_heads * pairs}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_power(e):
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_codes(x, e):
    """x (fp64) held in e4m3 under 2^e: to the nearest multiple of the step at its size, ties to even."""
    unit = _exact_power(e)
    y = x / unit
    step = _exact_power(torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 4)  # 2^size <= |y| < 2^(size + 1): steps of 2^(size - 3)
    return (torch.round(y / step) * step).clamp(-448, 448) * unit


def _exact_exponent(top):
    e = torch.frexp((top / 448).clamp(min=2.0 ** -90))[1] - 1  # 2^e <= top / 448 < 2^(e + 1), but for its rounding
    return torch.where(top <= 448 * _exact_power(e), e, e + 1).clamp(E_MIN, E_MAX)


def _exact_pages(pieces):
    """The values that one slot's pages hold after an append of each of `pieces` [heads, rows, 256], one behind the other: [heads, tokens, 256]."""
    heads, total = pieces[0].shape[0], sum(p.shape[1] for p in pieces)
    held = torch.zeros(heads, _pages(max(1, total)), PAGE, DIM, dtype=torch.float64, device=pieces[0].device)
    e = torch.full(held.shape[:2], E_MIN, device=held.device)
    at = 0
    for p in pieces:
        if p.shape[1]:
            lone = torch.zeros_like(held)
            lone.view(heads, -1, DIM)[:, at:at + p.shape[1]] = p.double()
            e = torch.maximum(e, _exact_exponent(lone.abs().amax((-2, -1))))
            held = _exact_codes(held + lone, e[..., None, None])
            at += p.shape[1]
    return held.flatten(1, 2)[:, :total]


def _exact_turn(case, x, at, weight):
    """x [heads, rows, 256] of one entry at positions `at` [rows], from the definition: pair by pair."""
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / DIM + EPS) * (1.0 + weight.double())
    out, n = y.clone(), case["rotary"] // 2
    for i in range(n):
        f = math.pow(BASE, -2.0 * i / (2 * n))
        grow = 1.0
        if case["scaling"] == "linear":
            f /= FACTOR
        elif case["scaling"] == "yarn":
            # the pair that makes r turns within the original length is number n ln(original / (2 pi r)) / ln base
            bounds = [n * math.log(ORIGINAL / (2 * math.pi * r)) / math.log(BASE) for r in (32.0, 1.0)]
            lo, hi = max(0, math.floor(bounds[0])), min(2 * n - 1, math.ceil(bounds[1]))
            part = min(1.0, max(0.0, (i - lo) / (hi - lo if hi > lo else 0.001)))
            f, grow = f * (1 - part) + f / FACTOR * part, 1.0 + 0.1 * math.log(FACTOR)
        elif case["scaling"] == "banded":
            length = 2 * math.pi / f
            if length > ORIGINAL:
                f /= FACTOR
            elif length > ORIGINAL / 4:
                keep = (ORIGINAL / length - 1) / 3
                f = keep * f + (1 - keep) * f / FACTOR
        c, s = torch.cos(at.double() * f) * grow, torch.sin(at.double() * f) * grow
        a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, n + i)
        out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., a] * s + y[..., b] * c
    return out


def exact(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kind, heads, rows = case["kind"], case["kv_heads"], case["rows"]
    if kind == "shared":
        parts = _history(g, case)
        q = _rows(g, case["groups"] * case["paths"], case["q_heads"], rows, "queries")
        common, branch = case["common"], case["branch"]
        tails, out = _tails(case), []
        for b, tail in enumerate(tails):
            k, v = (_exact_pages([parts[0][w][0, :, :common], parts[1][w][b // case["paths"], :, :branch], parts[2][w][b, :, :tail]]) for w in (0, 1))
            total = k.shape[1]
            t = torch.arange(total, device="cuda")
            p = total - rows + torch.arange(rows, device="cuda")[:, None]
            see = (t <= p) & ((t > p - case["window"]) | (t < case["sinks"])) if case["window"] else t <= p
            s = torch.einsum("hrid,htd->hrit", q[b].double().view(heads, -1, rows, DIM), k) / math.sqrt(DIM)
            out.append(torch.einsum("hrit,htd->hrid", torch.softmax(s.masked_fill(~see, -math.inf), -1), v).flatten(0, 1))
        return torch.stack(out)
    if kind == "append":
        lens, counts = _lens(case["tokens"], case["spread"], case["entries"]), _counts(case)
        past = [_rows(g, case["entries"], heads, max(1, max(lens)), w) for w in ("keys", "values")]
    x, weights = _projected(g, case)
    ids = _ids(g, case) if kind == "rotate" and case["ids"] else None
    q, k, v = x.view(case["entries"], rows, -1, DIM).permute(0, 2, 1, 3).split([case["q_heads"], heads, heads], 1)
    got = ([], [], [])
    for b in range(case["entries"]):
        if kind == "rotate":
            at = ids[b] if ids is not None else case["start"] + torch.arange(rows, device="cuda")
            got[0].append(_exact_turn(case, q[b], at, weights[0]))
            got[1].append(_exact_turn(case, k[b], at, weights[1]))
            continue
        n, t = counts[b], lens[b]
        at = t + torch.arange(n, device="cuda")
        turned = torch.zeros(case["q_heads"], rows, DIM, dtype=torch.float64, device="cuda")
        turned[:, :n] = _exact_turn(case, q[b, :, :n], at, weights[0])
        got[0].append(turned)
        for w, new in ((0, _exact_turn(case, k[b, :, :n], at, weights[1])), (1, v[b, :, :n])):
            held = _exact_pages([past[w][b, :, :t], new])[:, t - t % PAGE:]
            seen = torch.zeros(heads, rows + PAGE, DIM, dtype=torch.float64, device="cuda")
            seen[:, : held.shape[1]] = held
            got[1 + w].append(seen)
    return tuple(torch.stack(x) for x in got if x)
