"""Calls of both caches that feed one another on one stream, with nothing in
between: every kernel is launched behind the one before it and may start while
that one still writes, so each has to wait before it reads what it is given.
Each chain runs again with a synchronisation behind every call; the results
have to be the same, bit for bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def rows(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, 256, generator=g).bfloat16().cuda()


def paged(slots, H, tokens, seed):
    from rotated_bit_quantized_gb300 import IQPagedCache
    c = IQPagedCache(slots, H, slots * (tokens // 64 + 3))
    c.append(rows(seed, slots, H, tokens), rows(seed + 1, slots, H, tokens))
    return c


def rotated(slots, H, tokens, seed):
    from rotated_bit_quantized_gb300 import IQCache, Rotation
    rot = Rotation(0, 256, torch.device("cuda:0"))
    c = IQCache(slots, H, capacity=(tokens + 2304) // 256 * 256, device="cuda:0")
    c.append(rows(seed, slots, H, tokens), rows(seed + 1, slots, H, tokens), rot)
    return c, rot


def both_ways(chain, times=20):
    """chain(wait) runs the calls with wait() behind each; its results without waiting, against those with."""
    want = chain(torch.cuda.synchronize)
    for _ in range(times):
        got = chain(lambda: None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("slots,H,tokens,n", [(1, 2, 3000, 1), (8, 2, 9000, 1), (2, 2, 4000, 3), (1, 1, 6000, 130)])
def test_paged_results_are_the_rotated_caches_queries(slots, H, tokens, n):
    p = paged(slots, H, tokens, 1)
    c, rot = rotated(slots, H, 2000, 3)
    q = rows(5, slots, 8 * H if n <= 3 else 4 * H, n)

    def chain(wait):
        a = p.attend(q)
        wait()
        b = c.attend(a, rot)
        wait()
        d = p.attend(b)
        wait()
        return a, b, d, c.attend(d, rot)
    both_ways(chain)


@pytest.mark.parametrize("slots,H,tokens", [(1, 2, 500), (16, 2, 3000)])
def test_rows_read_from_pages_are_appended_and_attended(slots, H, tokens):
    """The rows that the paged cache hands out go straight into the other cache, fused with its attention and apart."""
    p = paged(slots, H, tokens, 1)
    c, rot = rotated(slots, H, 1920, 3)
    q = rows(5, slots, 4 * H, 1)

    def chain(wait):
        out = []
        for i in range(4):
            k, v = p.read(tokens // 2 + i, 1)
            wait()
            out.append(c.append_attend(k, v, q, rot))
            wait()
        k, v = p.read(3, 300)
        wait()
        c.append(k, v, rot)
        wait()
        out.append(c.attend(q, rot))
        c.trim(304)
        return out
    both_ways(chain)


@pytest.mark.parametrize("n", [1, 2])
def test_results_are_the_same_caches_next_queries(n):
    c, rot = rotated(8, 2, 9000, 3)
    q = rows(5, 8, 8, n)

    def chain(wait):
        out = [q]
        for _ in range(6):
            out.append(c.attend(out[-1], rot))
            wait()
        return out
    both_ways(chain)


def test_a_mask_made_by_the_call_before():
    """The mask's first bytes come from an attention that is still running."""
    c, rot = rotated(2, 2, 2048, 3)
    p = paged(2, 2, 5000, 1)
    q = rows(5, 2, 8, 2)

    def chain(wait):
        out = torch.zeros(2, 8, 2, 256, device="cuda")
        p.attend(q, out=out)
        wait()
        mask = out.view(-1)[: 2 * 2 * 2048].view(2, 2, 2048)
        return out, c.attend(q, rot, mask=mask)
    both_ways(chain)


@pytest.mark.parametrize("slots,H", [(1, 1), (1, 2), (3, 2)])
def test_an_appended_chunk_is_attended_at_once(slots, H):
    """A chunk whose attention encodes its own rows, then a step that reads all of them."""
    c, rot = rotated(slots, H, 256, 3)
    k, v, big = rows(7, slots, H, 1024), rows(8, slots, H, 1024), rows(9, slots, 8 * H, 1024)
    k1, v1, q1 = rows(10, slots, H, 1), rows(11, slots, H, 1), rows(12, slots, 8 * H, 1)

    def chain(wait):
        a = c.append_attend(k, v, big, rot)
        wait()
        b = c.append_attend(k1, v1, q1, rot)
        wait()
        d = c.attend(q1, rot)
        c.trim(1025)
        return a, b, d
    both_ways(chain)


def test_a_capture_in_between_does_not_count():
    """Calls captured between a call and the one that takes its result do not run there."""
    p = paged(4, 2, 9000, 1)
    c, rot = rotated(4, 2, 2000, 3)
    q, other = rows(5, 4, 16, 1), rows(6, 4, 16, 1)
    stream = torch.cuda.Stream()
    graphs = []

    def chain(wait):
        with torch.cuda.stream(stream):
            a = p.attend(q)
            wait()
            g = torch.cuda.CUDAGraph()
            g.capture_begin()
            p.attend(other)
            g.capture_end()
            graphs.append(g)
            return a, c.attend(a, rot)
    torch.cuda.synchronize()
    both_ways(chain, times=5)
