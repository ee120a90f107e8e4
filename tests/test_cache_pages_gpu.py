"""The cache's pages on the GPU against the same operations on Python lists: tables, lengths,
reference counts and every byte of the pages are equal."""
import random

import pytest
import torch

import exact_attention_103_b200 as ea
import serve_ref as ref

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Pair:
    """A cache and the lists that follow it."""

    def __init__(self, slots, max_pages, pages, page, layers=2, heads=2, d=64, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.c = ea.KVCache.empty(layers, pages, page, heads, d, slots, max_pages, dtype=dtype)
        for t in (self.c.k, self.c.v):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda").to(dtype))
        self.b = ref.Book(slots, max_pages, pages, page, [self.bits(t).clone() for t in (self.c.k, self.c.v)])

    @staticmethod
    def bits(t):
        return t.view(torch.uint8)

    def same(self):
        assert self.c.page_table.tolist() == self.b.table
        assert self.c.lens.tolist() == self.b.lens
        assert self.c.refs.tolist() == self.b.refs
        for t, w in zip((self.c.k, self.c.v), self.b.data):
            assert torch.equal(self.bits(t), w)

    def alloc(self, slots, want):
        assert self.c.alloc(ints(slots), ints(want)).tolist() == self.b.alloc(slots, want)

    def free(self, slots):
        self.c.free(ints(slots))
        self.b.free(slots)

    def fork(self, src, dst):
        assert self.c.fork(ints(src), ints(dst)).tolist() == self.b.fork(src, dst)

    def compact(self, drafted, path, slots, width=None, accepted=None):
        cu = [0]
        for n in drafted:
            cu.append(cu[-1] + n)
        accepted = accepted or [len(p) for p in path]
        width = width or max([1] + [len(p) for p in path])
        grid = [list(p) + [-1] * (width - len(p)) for p in path]
        self.c.compact(ints(cu), ints(grid), ints(accepted), slots=None if slots is None else ints(slots))
        self.b.compact(cu, grid, accepted, list(range(len(path))) if slots is None else slots)


@pytest.mark.parametrize("page,layers,heads,d,dtype", [
    (16, 1, 1, 64, torch.bfloat16), (64, 3, 4, 128, torch.bfloat16), (32, 2, 3, 64, torch.float8_e4m3fn)])
def test_random_histories(page, layers, heads, d, dtype):
    r = random.Random(page)
    p = Pair(20, 6, 70, page, layers, heads, d, dtype, seed=page)
    for step in range(60):
        kind = r.choice(["alloc", "alloc", "free", "fork", "compact"])
        empty = [s for s in range(20) if p.b.lens[s] == 0]
        held = [s for s in range(20) if p.b.lens[s] > 0]
        if kind == "alloc":
            slots = r.sample(range(20), r.randint(1, 8))
            p.alloc(slots, [min(6 * page, p.b.lens[s] + r.randint(0, 3 * page)) for s in slots])
        elif kind == "free" and held:
            p.free(r.sample(held, r.randint(1, min(4, len(held)))))
        elif kind == "fork" and held and empty:
            n = r.randint(1, len(empty))
            p.fork([r.choice(held) for _ in range(n)], r.sample(empty, n))
        elif kind == "compact" and held:
            # only tokens that the slot alone holds may be drafted: its last, partial page
            slots = r.sample(held, r.randint(1, min(5, len(held))))
            drafted = [r.randint(0, p.b.lens[s] % page) for s in slots]
            path = [sorted(r.sample(range(n), r.randint(0, n))) for n in drafted]
            p.compact(drafted, path, slots)
        p.same()
    ea.get_device_status()


def test_drafts_across_pages_and_many():
    """Drafted tokens over several pages, more accepted than a block moves together, none, all."""
    p = Pair(6, 40, 200, 16, layers=2, heads=3, d=128)
    p.alloc([0, 1, 2, 3, 5], [30, 16, 1, 0, 7])
    drafted = [300, 64, 17, 5, 0]
    p.alloc([0, 1, 2, 3, 5], [330, 80, 18, 5, 7])
    r = random.Random(2)
    path = [sorted(r.sample(range(300), 260)), [63], list(range(17)), [], []]
    p.compact(drafted, path, [0, 1, 2, 3, 5])
    p.same()
    ea.get_device_status()


def test_grants_in_order_when_pages_run_out():
    p = Pair(8, 10, 12, 16)
    p.alloc([3, 1], [16 * 5, 33])  # 5 + 3 pages: 4 left
    p.alloc([0, 2, 4, 1, 5], [32, 16 * 3, 16, 40, 1])  # 2 fit; 3 do not, nor what comes behind; 40 needs none
    assert p.b.lens == [32, 40, 0, 80, 0, 0, 0, 0]
    p.same()
    p.fork([1, 3, 1, 1, 1], [2, 4, 5, 6, 7])  # two free pages: the third partial copy and those behind wait
    assert p.b.lens[6:] == [0, 0] and p.b.lens[4] == 80
    p.same()
    p.free([3, 4])
    p.same()
    ea.get_device_status()


def test_refused_requests_leave_the_rest():
    p = Pair(5, 4, 16, 16)
    p.alloc([0, 1], [20, 20])
    for call in (lambda: p.alloc([2, 2, 7, -1, 3], [5, 50, 5, 5, 5]),   # named twice; out of range
                 lambda: p.alloc([0, 3], [10, 65]),                     # shorter; beyond max_pages
                 lambda: p.fork([0, 0, 1, 9], [4, 4, 1, 3]),            # twice; onto itself; bad source
                 lambda: p.fork([0], [1]),                              # not empty
                 lambda: p.free([-3, 77, 4]),
                 lambda: p.compact([3, 25, 2], [[0, 0], [1], [1]], [0, 1, 2]),  # not increasing; more than it holds
                 lambda: p.compact([3, 3], [[0, 3], [1]], [0, 0]),      # beyond the drafts; slot named twice
                 lambda: p.compact([3], [[0]], [5]),
                 lambda: p.compact([3], [[0]], [0], accepted=[4])):
        call()
        p.same()
        with pytest.raises(ea.AttnError) as e:
            ea.get_device_status()
        assert e.value.status == ea.ATTN_ERR_INVALID_ARG
    p.free([0, 0, 0])  # the same slot again is a no-op
    p.same()
    ea.get_device_status()


def test_compact_leaves_shared_pages_alone():
    """Drafted tokens in a full page that a fork shares: nothing moves; kept in place, they may stay."""
    p = Pair(4, 4, 16, 16)
    p.alloc([0, 1], [32, 20])
    p.fork([0], [2])
    p.c.compact(ints([0, 6, 9]), ints([[2, 4], [1, -1]]), ints([2, 1]), slots=ints([0, 1]))
    p.b.compact([0, 0, 3], [[-1], [1]], [0, 1], [0, 1])  # slot 1's token moves in its own page
    p.same()
    with pytest.raises(ea.AttnError):
        ea.get_device_status()
    p.compact([6], [[0, 1, 2]], [2])
    p.same()
    ea.get_device_status()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
def test_offsets_beyond_31_bits(dtype):
    """Pages whose first value has an index above 2^31, and above 2^32 in bytes, in the second layer."""
    layers, pages, page, heads, d = 2, 70000, 16, 8, 128
    c = ea.KVCache.empty(layers, pages, page, heads, d, 4, 8, dtype=dtype)
    assert c.k[1, -40:].storage_offset() > 2 ** 31
    c.refs[:-40] = 1
    lens = [50, 33, 128]
    assert c.alloc(ints([0, 1, 2]), ints(lens)).tolist() == [1, 1, 1]
    assert c.page_table[:3].max() >= pages - 40 and c.page_table[0].tolist()[:4] == list(range(pages - 40, pages - 36))
    g = torch.Generator(device="cuda").manual_seed(1)
    T = sum(lens)
    k, v = (torch.randn((T, heads, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn((T, heads, d), generator=g, device="cuda").to(torch.bfloat16)
    cu = ints([0, 50, 83, 211])
    for layer in range(layers):
        ea.rope_append(c, None, k, v, cu, layer=layer)
    assert torch.equal(c.k[1, pages - 40].view(torch.uint8), k[:16].to(dtype).view(torch.uint8))
    o, lse = ea.tree_fwd(c, q, cu, layer=1)
    small = ea.KVCache.empty(1, 16, page, heads, d, 4, 8, dtype=dtype)
    small.alloc(ints([0, 1, 2]), ints(lens))
    ea.rope_append(small, None, k, v, cu)
    want = ea.tree_fwd(small, q, cu)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    # token 45 of slot 0 takes the place of token 40, then a fork copies the tail
    c.compact(ints([0, 10]), ints([[5]]), ints([1]), slots=ints([0]))
    assert c.fork(ints([0]), ints([3])).tolist() == [1]
    assert c.lens.tolist() == [41, 33, 128, 41]
    for t, x in ((c.k, k), (c.v, v)):
        for s in (0, 3):
            got = t[1, int(c.page_table[s, 2])].view(torch.uint8)
            rows = x[list(range(32, 40)) + [45]].to(dtype).view(torch.uint8)
            assert torch.equal(got[:9], rows)
    c.copy(ints([int(c.page_table[0, 0])]), ints([pages - 1]))
    assert torch.equal(c.v[1, pages - 1].view(torch.uint8), v[:16].to(dtype).view(torch.uint8))
    ea.get_device_status()


def test_compact_defaults_to_the_first_slots():
    p = Pair(3, 4, 16, 16)
    p.alloc([0, 1, 2], [20, 33, 5])
    p.compact([4, 2], [[1, 3], [0]], None, width=5)
    p.same()
    ea.get_device_status()


@pytest.mark.parametrize("page,heads,d,layers,n", [(16, 1, 64, 1, 3), (16, 8, 128, 3, 700), (128, 5, 128, 2, 9), (1024, 1, 64, 2, 2)])
def test_copy(page, heads, d, layers, n):
    pages = 2 * n + 3
    p = Pair(1, 1, pages, page, layers, heads, d)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(n)).tolist()
    src, dst = order[:n], order[n:2 * n]
    src[-1] = src[0]  # one page to two places
    p.c.copy(ints(src), ints(dst))
    for t in p.b.data:
        t[:, dst] = t[:, src]
    p.same()
    ea.get_device_status()


def test_copy_names_twice_and_refuses():
    p = Pair(1, 1, 10, 16)
    p.c.copy(ints([0, 1, 2, 5]), ints([6, 6, 7, 5]))  # 6 named twice: the last counts; 5 onto itself
    for t in p.b.data:
        t[:, 6], t[:, 7] = t[:, 1], t[:, 2]
    p.same()
    ea.get_device_status()
    p.c.copy(ints([0, 8, 10, 3]), ints([8, 9, 1, -1]))  # 8 is read and written; numbers out of range
    for t in p.b.data:
        t[:, 8] = t[:, 0]
    p.same()
    with pytest.raises(ea.AttnError):
        ea.get_device_status()


def test_large_pool_many_requests():
    """Thousands of requests over a pool larger than one stretch of the search."""
    r = random.Random(4)
    p = Pair(5000, 9, 40001, 16, layers=1, heads=1)
    slots = r.sample(range(5000), 4000)
    p.alloc(slots, [r.randint(0, 144) for _ in slots])
    p.free(r.sample(slots, 1500))
    p.alloc(list(range(5000)), [max(p.b.lens[s], r.randint(0, 100)) for s in range(5000)])
    p.same()
    ea.get_device_status()
