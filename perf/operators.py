"""The paged 8-bit cache's operators as a user's program calls them, and their plain forms.

The cache: pages of 64 tokens for all kv heads, head_dim 256, codes in e4m3 with one power-of-two
scale per page and head (keys and values apart), one row of page ids per sequence slot.

kind        one pass
"append"    new rows of every slot quantised into its pages, then read back as the values held
"attend"    attention of the queries over every slot's pages (causal; window > 0: only the last `window`
            positions and the first `sinks` tokens are visible)
"fork"      one prompt forked to `slots` paths that share its pages, one step on each (rows appended, which
            copies the shared last page, then attended), and the new rows read back
"compact"   the live pages of a pool copied into a tight one, each distinct page once, in slot order
"""
import math

import torch

own = False

PAGE, DIM, E_MIN, E_MAX, TOP = 64, 256, -40, 60, 448.0


def listed():
    def case(name, kind, slots, tokens, rows, *, q_heads=16, kv_heads=2, spread=0, window=0, sinks=0):
        return {"name": name, "kind": kind, "slots": slots, "tokens": tokens, "spread": spread, "rows": rows,
                "q_heads": q_heads, "kv_heads": kv_heads, "window": window, "sinks": sinks}

    return [
        # one generated token for each of 32 sequences at lengths of their own: latency
        case("append_step", "append", 32, 2000, 1, spread=1500),
        # a batch of prompt chunks, the benchmark's append shape
        case("append_prompts", "append", 32, 0, 4096),
        # one user, one token, a short history: the smallest call of a chat
        case("decode_single", "attend", 1, 4096, 1),
        # the benchmark's batched decode: 32 histories of 32768 tokens
        case("decode_batch", "attend", 32, 32768, 1),
        # continuous batching: lengths from one token to 20000, few of them alike, other head counts
        case("decode_ragged", "attend", 23, 10001, 1, spread=10000, q_heads=12, kv_heads=4),
        # speculative verify: four drafted tokens against long histories
        case("verify_long", "attend", 8, 131072, 4),
        # the last chunk of a chunked prefill: 2048 queries, their own rows already appended
        case("prefill_chunk", "attend", 1, 32768, 2048),
        # a batch of prompts of an odd length, each attending to itself
        case("prefill_prompts", "attend", 4, 1531, 1531),
        # decode with a sliding window and four sinks over long histories
        case("window_decode", "attend", 32, 32768, 1, window=4096, sinks=4),
        # a long prompt under a window of odd size and a few sinks, in one call
        case("window_prompt", "attend", 1, 8191, 8191, window=1023, sinks=16),
        # a prompt tried along 32 paths, one token each; its last page is partly full
        case("fork_paths", "fork", 32, 4109, 1),
        # a pool of forked, partly released sequences moved into a tight one
        case("compact_pool", "compact", 24, 16300, 1, spread=500),
    ]


def _between(rng, low, high):
    """An odd or even whole number, spread over its logarithm."""
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high + 0.5))))))


def draw(rng):
    kind = rng.choice(["append", "append", "attend", "attend", "attend", "attend", "window", "window", "fork", "compact"])
    kv_heads = rng.choice([1, 2, 4, 8])
    q_heads = kv_heads * rng.choice([1, 2, 3, 4, 6, 8])
    case = {"kind": "attend" if kind == "window" else kind, "q_heads": q_heads, "kv_heads": kv_heads, "window": 0, "sinks": 0, "spread": 0}
    if kind == "append":
        slots = _between(rng, 1, 48)
        rows = _between(rng, 1, max(1, 262144 // (slots * kv_heads)))
        tokens = rng.randrange(0, 3000)
        return case | {"slots": slots, "tokens": tokens, "spread": tokens // 2, "rows": rows}
    if kind == "fork":
        return case | {"slots": _between(rng, 2, 64), "tokens": _between(rng, 1, 8000), "rows": rng.choice([1, 1, 2, 5])}
    if kind == "compact":
        slots = _between(rng, 3, 40)
        tokens = _between(rng, 64, max(65, 700000 // (slots * kv_heads)))
        return case | {"slots": slots, "tokens": tokens, "spread": tokens // 4, "rows": 1}
    if kind == "window":
        case |= {"window": _between(rng, 1, 6000), "sinks": rng.choice([0, 1, 4, 16, 70])}
    rows = rng.choice([1, 1, 1, 2, 4, 5, _between(rng, 6, 3000)])
    if rows <= 5:  # decode and verify: bounded by the tokens held
        slots = _between(rng, 1, 64)
        tokens = _between(rng, rows, min(150000, 1900000 // (slots * kv_heads)))
    else:  # prompts and chunks: bounded by the pairs
        slots = rng.choice([1, 1, 2, 3, 5])
        most = min(60000, 60 * 10 ** 6 * 16 // (slots * rows * q_heads))
        tokens = _between(rng, rows, max(rows, most))
    return case | {"slots": slots, "tokens": tokens, "spread": (tokens - rows) // 2, "rows": rows}


# ------------------------------------------------------------------ inputs

def _lens(case, n):
    """The slots' lengths: `tokens`, give or take `spread`, the same for every seed; the first the shortest."""
    s = case["spread"]
    return [case["tokens"] - s + (2 * s * ((7 * b) % n)) // max(1, n - 1) for b in range(n)]


def _rows(g, lead, heads, rows, kind):
    """bf16 rows [lead, heads, rows, 256]: standard normals; keys have eight channels per head twenty times as large."""
    x = torch.randn(lead, heads, rows, DIM, generator=g, device="cuda")
    if kind == "keys":
        at = torch.rand(lead, heads, 1, DIM, generator=g, device="cuda").topk(8, dim=-1).indices
        x.scatter_(-1, at.expand(-1, -1, rows, -1), 20.0 * x.gather(-1, at.expand(-1, -1, rows, -1)))
    return x.to(torch.bfloat16)


def _pages(tokens):
    return (tokens + PAGE - 1) // PAGE


def _forks(case):
    """What happened to a "compact" pool: every third slot was forked from the one before it, every fifth released."""
    n = case["slots"]
    return [b for b in range(n) if b % 3 == 2], [b for b in range(n) if b % 5 == 4]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kind, heads, rows = case["kind"], case["kv_heads"], case["rows"]
    n = 1 if kind == "fork" else case["slots"]
    lens = _lens(case, n)
    st = {"case": case, "scale": 1.0 / math.sqrt(DIM)}
    slots = case["slots"] + 1 if kind == "fork" else case["slots"]
    room = rows if kind in ("append", "fork") else 0
    pages = sum(_pages(t + room) for t in lens)
    if kind == "fork":
        pages += case["slots"] * (1 + _pages(rows))
    longest = max(lens) + room
    # the history, appended once; the lengths differ, so rows past a slot's own are padding
    past_k, past_v = (_rows(g, n, heads, max(1, max(lens)), w) for w in ("keys", "values"))
    # the handle that a program keeps: the framework's cache where own is true, plain tensors of the same layout else
    if own:
        from rotated_bit_quantized_gb300 import IQPagedCache

        st["cache"] = cache = IQPagedCache(slots, heads, pages, max_tokens=longest)
        cache.append(past_k, past_v, slots=range(n), counts=lens)
    else:
        st["pool"] = pool = _new_pool(slots, heads, pages, _pages(longest))
        _plain_append(pool, past_k, past_v, torch.arange(n, device="cuda"), torch.tensor(lens, device="cuda"))
    if kind == "compact":
        forked, released = _forks(case)
        if own:
            cache.fork([b - 1 for b in forked], forked)
            cache.free(released)
            st["into"] = IQPagedCache(slots, heads, cache.pages_used, max_tokens=longest)
        else:
            pool["table"][forked], pool["lens"][forked] = pool["table"][[b - 1 for b in forked]], pool["lens"][[b - 1 for b in forked]]
            pool["lens"][released] = 0
        return st
    lead = case["slots"]
    if kind in ("append", "fork"):
        st["keys"], st["values"] = (_rows(g, lead, heads, rows, w) for w in ("keys", "values"))
        st["at"] = lens if kind == "append" else lens * lead
    if kind in ("attend", "fork"):
        st["q"] = _rows(g, lead, case["q_heads"], rows, "queries")
    return st


# ------------------------------------------------------------------ one pass

def run(state):
    return _own(state) if own else _plain(state)


def _own(st):
    case, cache = st["case"], st["cache"]
    kind, rows = case["kind"], case["rows"]
    if kind == "append":
        cache.trim(cache.lens - st["at"])
        cache.append(st["keys"], st["values"])
        return cache.read(st["at"], rows)
    if kind == "attend":
        return cache.attend(st["q"], scale=st["scale"], window=case["window"], sinks=case["sinks"])
    if kind == "fork":
        paths = range(1, case["slots"] + 1)
        cache.fork([0] * case["slots"], paths)
        out = cache.append_attend(st["keys"], st["values"], st["q"], scale=st["scale"], slots=paths)
        return out, cache.read(st["at"], rows, slots=paths)
    to = cache.compact(out=st["into"])
    f8 = torch.float8_e4m3fn
    return to.k_codes.view(f8), to.v_codes.view(f8), to.k_scales, to.v_scales, torch.from_numpy(to.lens)


def _plain(st):
    case, pool = st["case"], st["pool"]
    kind, rows = case["kind"], case["rows"]
    everyone = torch.arange(case["slots"], device="cuda")
    if kind == "append":
        at = torch.tensor(st["at"], device="cuda")
        pool["lens"][:] = at
        _plain_append(pool, st["keys"], st["values"], everyone, torch.full_like(at, rows))
        return _plain_read(pool, everyone, at, rows)
    if kind == "attend":
        return _plain_attend(pool, st["q"], everyone, st["scale"], case["window"], case["sinks"])
    if kind == "fork":
        paths, at = everyone + 1, torch.tensor(st["at"], device="cuda")
        pool["table"][paths], pool["lens"][paths] = pool["table"][0].clone(), pool["lens"][0].clone()
        _plain_append(pool, st["keys"], st["values"], paths, torch.full_like(at, rows), first=_pages(case["tokens"]))
        out = _plain_attend(pool, st["q"], paths, st["scale"], 0, 0)
        return out, _plain_read(pool, paths, at, rows)
    # compact: distinct live pages in the order of their first visit
    live = torch.arange(pool["table"].shape[1], device="cuda") < ((pool["lens"] + PAGE - 1) // PAGE)[:, None]
    seen = pool["table"][live]
    order = torch.full((pool["k"].shape[0],), seen.numel(), device="cuda").scatter_reduce(0, seen, torch.arange(seen.numel(), device="cuda"), "amin")
    ids = torch.argsort(order, stable=True)[: int((order < seen.numel()).sum())]
    f8 = torch.float8_e4m3fn
    return pool["k"][ids].view(f8), pool["v"][ids].view(f8), pool["ks"][ids], pool["vs"][ids], pool["lens"].to(torch.int32).cpu()


# ------------------------------------------------------------------ plain forms

def _new_pool(slots, heads, pages, width):
    dev = "cuda"
    return {"k": torch.zeros(pages, heads, PAGE, DIM, dtype=torch.uint8, device=dev), "v": torch.zeros(pages, heads, PAGE, DIM, dtype=torch.uint8, device=dev),
            "ks": torch.ones(pages, heads, device=dev), "vs": torch.ones(pages, heads, device=dev),
            "table": torch.zeros(slots, width, dtype=torch.int64, device=dev), "lens": torch.zeros(slots, dtype=torch.int64, device=dev)}


def _exponent(top):
    """The least e with top <= 448 * 2^e, within its limits."""
    m, x = torch.frexp(top)  # top = m * 2^x, 0.5 <= m < 1;  448 = 0.875 * 2^9
    return torch.where(top > 0, x - 9 + (m > 0.875).int(), torch.full_like(x, E_MIN)).clamp(E_MIN, E_MAX)


def _power(e):
    """2^e in fp32, bit by bit: a power function need not be exact."""
    return ((e + 127) << 23).view(torch.float32)


def _held(codes, scales):
    return codes.view(torch.float8_e4m3fn).float() * scales[..., None, None]


def _plain_append(pool, keys, values, slots, counts, first=None):
    """Rows i < counts[b] of keys / values [b] go behind what slot slots[b] holds. Slot b's fresh pages are taken in
    order behind all pages in use, or, for forked slots, behind the `first` shared ones, whose last, partly full one is copied."""
    lead, heads, n = keys.shape[:3]
    at = pool["lens"][slots]
    inside = at % PAGE
    width = (PAGE - 1 + n + PAGE - 1) // PAGE
    # which pages each slot writes, their ids
    index = at[:, None] // PAGE + torch.arange(width, device="cuda")
    used = (inside + counts + PAGE - 1) // PAGE
    written = torch.arange(width, device="cuda") < torch.where(counts > 0, used, 0)[:, None]
    had = index < ((at + PAGE - 1) // PAGE)[:, None]  # only the first can be there already, partly full
    index_in = index.clamp(max=pool["table"].shape[1] - 1)
    held = pool["table"][slots[:, None], index_in]
    if first is None:
        new = written & ~had
        base = ((pool["lens"] + PAGE - 1) // PAGE).sum()
    else:
        new, base = written, torch.tensor(first, device="cuda")
    ids = torch.where(new, base + new.flatten().cumsum(0).view_as(new) - 1, held)
    # old and new rows side by side: [lead, heads, width * 64, 256]
    place = inside[:, None] + torch.arange(n, device="cuda")
    valid = torch.arange(n, device="cuda") < counts[:, None]
    place = torch.where(valid, place, width * PAGE)
    old_rows = torch.arange(PAGE, device="cuda") < inside[:, None]
    for x, codes, scales in ((keys, pool["k"], pool["ks"]), (values, pool["v"], pool["vs"])):
        fresh = torch.zeros(lead, heads, width * PAGE + 1, DIM, device="cuda")
        fresh.scatter_(2, place[:, None, :, None].expand(-1, heads, -1, DIM), x.float())
        fresh = fresh[:, :, :-1].reshape(lead, heads, width, PAGE, DIM)
        e = _exponent(fresh.abs().amax((-2, -1)))
        first_e = torch.frexp(scales[held[:, 0]])[1] - 1
        e[:, :, 0] = torch.where((inside > 0)[:, None], torch.maximum(e[:, :, 0], first_e), e[:, :, 0])
        fresh[:, :, 0] += torch.where(old_rows[:, None, :, None], _held(codes[held[:, 0]], scales[held[:, 0]]), 0.0)
        scale = _power(e)
        c = (fresh / scale[..., None, None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn).view(torch.uint8)
        codes[ids[written]] = c.transpose(1, 2)[written]
        scales[ids[written]] = scale.transpose(1, 2)[written]
    row, col = written.nonzero(as_tuple=True)
    pool["table"][slots[row], index[row, col]] = ids[row, col]
    pool["lens"][slots] = at + counts


def _plain_values(pool, slots, width):
    """The values held by the first `width` pages of the slots: keys, values [slots, heads, width * 64, 256], fp32."""
    ids = pool["table"][slots, :width]
    return [_held(c[ids], s[ids]).transpose(1, 2).reshape(len(slots), c.shape[1], width * PAGE, DIM) for c, s in ((pool["k"], pool["ks"]), (pool["v"], pool["vs"]))]


def _plain_read(pool, slots, start, n):
    place = start[:, None] + torch.arange(n, device="cuda")
    live = place < pool["lens"][slots][:, None]
    ids = pool["table"][slots[:, None], (place // PAGE).clamp(max=pool["table"].shape[1] - 1)]
    out = []
    for c, s in ((pool["k"], pool["ks"]), (pool["v"], pool["vs"])):
        rows = c[ids, :, place % PAGE].view(torch.float8_e4m3fn).float() * s[ids][..., None]  # [slots, n, heads, 256]
        out.append(torch.where(live[:, :, None, None], rows, 0.0).transpose(1, 2).to(torch.bfloat16))
    return out


def _visible(lens, n, width, window, sinks):
    """[slots, n, width]: the keys that each query sees."""
    key = torch.arange(width, device=lens.device)
    at = (lens[:, None] - n + torch.arange(n, device=lens.device))[:, :, None]
    see = key <= at
    return see & ((key > at - window) | (key < sinks)) if window else see


def _plain_attend(pool, q, slots, scale, window, sinks):
    lead, q_heads, n, _ = q.shape
    heads = pool["k"].shape[1]
    width = pool["table"].shape[1]
    k, v = _plain_values(pool, slots, width)
    rep = q_heads // heads
    s = (q.float().view(lead, heads, rep * n, DIM) @ k.transpose(-1, -2)).mul_(scale).view(lead, heads, rep, n, width * PAGE)
    see = _visible(pool["lens"][slots], n, width * PAGE, window, sinks)[:, None, None]
    s.masked_fill_(~see, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(top.isfinite(), top, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.view(lead, heads, rep * n, width * PAGE) @ v).view(lead, heads, rep, n, DIM)
    return torch.where(total > 0, out / total, 0.0).view(lead, q_heads, n, DIM).to(torch.bfloat16)


# ------------------------------------------------------------------ work

def _pairs(length, rows, window, sinks):
    """(visible pairs of one head, keys that some query sees) of `rows` last queries over `length` keys."""
    pairs = 0
    for at in range(length - rows, length):
        low = max(0, at - window + 1) if window else 0
        pairs += at + 1 - low + min(sinks, low) if window else at + 1
    low = max(0, length - rows - window + 1) if window else 0
    return pairs, length - low + (min(sinks, low) if window else 0)


def work(case):
    kind, heads, rows = case["kind"], case["kv_heads"], case["rows"]
    lead, q_heads = case["slots"], case["q_heads"]
    appended = lead * heads * rows * (2 * 2 * DIM + 2 * DIM)  # rows in as bf16, out as codes
    back = lead * heads * rows * (2 * DIM + 2 * 2 * DIM)  # codes in, rows out as bf16
    asked = lead * q_heads * rows * 2 * 2 * DIM  # queries in, results out
    if kind == "append":
        return {"bytes": appended + back, "flops": 4 * lead * heads * rows * DIM}
    if kind == "attend":
        both = [_pairs(t, rows, case["window"], case["sinks"]) for t in _lens(case, lead)]
        return {"bytes": asked + 2 * DIM * heads * sum(k for _, k in both), "flops": 4 * DIM * q_heads * sum(p for p, _ in both)}
    if kind == "fork":
        t = case["tokens"]
        shared = 2 * DIM * heads * t  # the prompt's pages are the same for all paths
        copied = lead * 2 * DIM * heads * (t % PAGE)
        pairs, _ = _pairs(t + rows, rows, 0, 0)
        return {"bytes": appended + back + asked + shared + copied, "flops": 4 * DIM * q_heads * lead * pairs}
    forked, released = _forks(case)
    lens = _lens(case, lead)
    live = {b: (b - 1 if b in forked else b) for b in range(lead) if b not in released}
    pages = sum(_pages(lens[b]) for b in set(live.values()))
    return {"bytes": 2 * pages * heads * (2 * PAGE * DIM + 8), "flops": 0}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_codes(x, e):
    """x (fp64) held in e4m3 under 2^e: to the nearest multiple of the step at its size, ties to even."""
    unit = _exact_power(e)
    y = x / unit
    step = _exact_power(torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 4)  # 2^size <= |y| < 2^(size + 1): steps of 2^(size - 3)
    return (torch.round(y / step) * step).clamp(-448, 448) * unit


def _exact_power(e):
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_exponent(top):
    e = torch.frexp((top / 448).clamp(min=2.0 ** -90))[1] - 1  # 2^e <= top / 448 < 2^(e + 1), but for its rounding
    return torch.where(top <= 448 * _exact_power(e), e, e + 1).clamp(E_MIN, E_MAX)


def _exact_pages(x, length, more=None):
    """The values that a slot's pages hold after `length` rows of x [heads, rows, 256] and then the rows `more`:
    [heads, pages, 64, 256], and their exponents [heads, pages]."""
    heads = x.shape[0]
    total = length + (0 if more is None else more.shape[1])
    held = torch.zeros(heads, _pages(max(1, total)) * PAGE, DIM, dtype=torch.float64, device=x.device)
    if length:
        held[:, :length] = x[:, :length].double()
    paged = held.view(heads, -1, PAGE, DIM)
    e = _exact_exponent(paged.abs().amax((-2, -1)))
    paged.copy_(_exact_codes(paged, e[..., None, None]))
    if more is not None:
        lone = torch.zeros_like(held)
        lone[:, length:total] = more.double()
        lone = lone.view_as(paged)
        now = _exact_exponent(lone.abs().amax((-2, -1)))
        begun = torch.arange(now.shape[1], device=x.device) * PAGE < length
        e = torch.where(begun, torch.maximum(e, now), now)
        paged.copy_(_exact_codes(paged + lone, e[..., None, None]))
    return paged, e


def exact(case, seed):
    kind, heads, rows, lead = case["kind"], case["kv_heads"], case["rows"], case["slots"]
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = 1 if kind == "fork" else lead
    lens = _lens(case, n)
    past = [_rows(g, n, heads, max(1, max(lens)), w) for w in ("keys", "values")]
    new = [_rows(g, lead, heads, rows, w) for w in ("keys", "values")] if kind in ("append", "fork") else None
    q = _rows(g, lead, case["q_heads"], rows, "queries") if kind in ("attend", "fork") else None
    if kind == "compact":  # each live slot's own pages, in the order of the slots
        forked, released = _forks(case)
        live = [b - 1 if b in forked else b for b in range(lead) if b not in released]
        both = [[_exact_pages(x[b], lens[b]) for b in dict.fromkeys(live)] for x in past]
        codes = [torch.cat([(p / _exact_power(e)[..., None, None]).transpose(0, 1) for p, e in kv]) for kv in both]
        held = [0 if b in released else lens[b - 1] if b in forked else lens[b] for b in range(lead)]
        return codes + [torch.cat([_exact_power(e).transpose(0, 1) for _, e in kv]) for kv in both] + [torch.tensor(held, dtype=torch.int32)]
    out, back = [], ([], [])
    rep = case["q_heads"] // heads
    for b in range(lead):
        at = 0 if kind == "fork" else b
        k, v = (_exact_pages(x[at], lens[at], None if new is None else y[b])[0].flatten(1, 2)[:, :lens[at] + (0 if new is None else rows)]
                for x, y in zip(past, new or past))
        if new is not None:
            back[0].append(k[:, lens[at]:])
            back[1].append(v[:, lens[at]:])
        if q is None:
            continue
        result = torch.zeros(heads, rep, rows, DIM, dtype=torch.float64, device="cuda")
        for i in range(0, rows, 512):  # pieces of the queries, to bound the scores' memory
            part = q[b].double().view(heads, rep, rows, DIM)[:, :, i:i + 512]
            m = part.shape[2]
            s = torch.einsum("hrid,htd->hrit", part, k) / math.sqrt(DIM)
            t = torch.arange(k.shape[1], device="cuda")
            p = k.shape[1] - rows + i + torch.arange(m, device="cuda")[:, None]
            see = t <= p
            if case["window"]:
                see &= (t > p - case["window"]) | (t < case["sinks"])
            result[:, :, i:i + 512] = torch.einsum("hrit,htd->hrid", torch.softmax(s.masked_fill(~see, -math.inf), -1), v)
        out.append(result.view(heads * rep, rows, DIM))
    read = [torch.stack(x) for x in back] if new is not None else None
    if kind == "append":
        return read
    return torch.stack(out) if kind == "attend" else (torch.stack(out), read)
