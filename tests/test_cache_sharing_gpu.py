"""Slots that share pages: no operation on one slot changes the tokens of another."""
import pytest
import torch

import exact_attention_103_b200 as ea
import serve_ref as ref
import test_tree_gpu as tree

pytestmark = pytest.mark.gpu
ints = tree.ints


def cache(slots, max_pages, pages, page=16, layers=2, heads=2, d=64, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = ea.KVCache.empty(layers, pages, page, heads, d, slots, max_pages, dtype=dtype)
    for t in (c.k, c.v):
        t.copy_(torch.randn(t.shape, generator=g, device="cuda").to(dtype))
    return c


def tokens(c, slot):
    """The bytes of a slot's tokens in every layer."""
    row, n = c.page_table[slot].tolist(), int(c.lens[slot])
    return [ref.gather(t[l].view(torch.uint8), row, n, c.page_size).clone() for t in (c.k, c.v) for l in range(c.layers)]


def sound(c):
    """Counts are those of the holders; what is behind a slot's pages is not looked at."""
    held = torch.zeros_like(c.refs)
    for s in range(c.slots):
        for p in c.page_table[s, :-(-int(c.lens[s]) // c.page_size)].tolist():
            held[p] += 1
    assert torch.equal(c.refs, held)


def same(a, b, n=None):
    assert all(torch.equal(x[:n], y[:n]) for x, y in zip(a, b))


def grow(c, slots, lens, value):
    """alloc, then an append of the new tokens in every layer."""
    old = c.lens.tolist()
    new = [w - old[s] for s, w in zip(slots, lens)]
    assert c.alloc(ints(slots), ints(lens)).tolist() == [1] * len(slots)
    x = torch.full((sum(new), c.heads, c.d), value, device="cuda").to(torch.bfloat16)
    for l in range(c.layers):
        ea.rope_append(c, None, x, x, tree.cu_of(new), slots=ints(slots), layer=l)
    return new


@pytest.mark.parametrize("dtype,layers,heads,d", [(torch.bfloat16, 2, 2, 64), (torch.float8_e4m3fn, 3, 5, 128)])
def test_growing_behind_a_cut_inside_a_shared_page(dtype, layers, heads, d):
    """A slot whose drafts end inside a page that a fork holds too grows into a page of its own."""
    c = cache(4, 6, 20, layers=layers, heads=heads, d=d, dtype=dtype)
    c.alloc(ints([0]), ints([32]))
    c.fork(ints([0]), ints([2]))
    keep = tokens(c, 0)
    c.compact(ints([0, 6]), ints([[0, 1, 2]]), ints([3]), slots=ints([2]))  # 29 tokens, in place
    assert c.lens.tolist() == [32, 0, 29, 0]
    same(keep, tokens(c, 2), 29)
    grow(c, [2], [30], 3.0)
    same(keep, tokens(c, 0))
    same(keep, tokens(c, 2), 29)
    assert c.page_table[0, 0] == c.page_table[2, 0] and c.page_table[0, 1] != c.page_table[2, 1]
    sound(c)
    ea.get_device_status()


def test_both_holders_grow():
    """Cut to different ends in one page, grown in one call and in two; over several pages."""
    for calls in ([[0, 2]], [[0], [2]], [[2], [0]]):
        c = cache(4, 6, 20)
        c.alloc(ints([0, 1]), ints([48, 7]))
        c.fork(ints([0]), ints([2]))
        keep, other = tokens(c, 0), tokens(c, 1)
        c.compact(ints([0, 10, 20]), ints([[0, 1], [0, 1]]), ints([2, 1]), slots=ints([0, 2]))  # 40 and 39
        assert c.lens.tolist() == [40, 7, 39, 0]
        sound(c)
        for i, slots in enumerate(calls):
            grow(c, slots, [{0: 41, 2: 70}[s] for s in slots], 3.0 + i)
            sound(c)
        same(keep, tokens(c, 0), 40)
        same(keep, tokens(c, 2), 39)
        same(other, tokens(c, 1))
        pages = [p for s in (0, 2) for p in c.page_table[s, 2:-(-int(c.lens[s]) // 16)].tolist()]
        assert len(set(pages)) == len(pages)
        ea.get_device_status()


def test_without_a_page_for_the_copy():
    """Not granted, nothing changes; what needs no page is granted all the same."""
    c = cache(4, 6, 3)
    c.alloc(ints([0, 1]), ints([32, 3]))
    c.fork(ints([0]), ints([2]))
    c.compact(ints([0, 6]), ints([[0]]), ints([1]), slots=ints([2]))  # 27 of 32, shared
    state = [t.clone() for t in (c.page_table, c.lens, c.refs, c.k.view(torch.uint8), c.v.view(torch.uint8))]
    assert c.alloc(ints([2, 1]), ints([28, 4])).tolist() == [0, 1]
    state[1][1] = 4
    for x, y in zip(state, (c.page_table, c.lens, c.refs, c.k.view(torch.uint8), c.v.view(torch.uint8))):
        assert torch.equal(x, y)
    assert c.alloc(ints([2]), ints([27])).tolist() == [1]  # nothing to grow: nothing to copy
    assert torch.equal(c.refs, state[2])
    c.free(ints([1]))
    assert c.alloc(ints([2]), ints([28])).tolist() == [1]
    assert c.page_table[2, 1] == state[0][1, 0] and c.refs.tolist() == [2, 1, 1]
    ea.get_device_status()


def test_many_slots_of_one_page():
    """Forty forks cut inside the page they share, grown together: pages in order of the requests."""
    n = 40
    c = cache(n + 1, 4, 100, layers=3)
    c.alloc(ints([0]), ints([32]))
    c.fork(ints([0] * n), ints(list(range(1, n + 1))))
    keep = tokens(c, 0)
    drafted = [1 + s % 15 for s in range(1, n + 1)]
    c.compact(tree.cu_of(drafted), ints([[-1]] * n), ints([0] * n), slots=ints(list(range(1, n + 1))))
    sound(c)
    lens = c.lens.tolist()
    grow(c, list(range(n, 0, -1)), [lens[s] + 1 + s % 30 for s in range(n, 0, -1)], 5.0)
    sound(c)
    same(keep, tokens(c, 0))
    for s in range(1, n + 1):
        same(keep, tokens(c, s), lens[s])
        assert all((x[lens[s]:] != 0).any() for x in tokens(c, s))
    ea.get_device_status()


@pytest.mark.parametrize("fill", [0, 1, 30, 200, 1000])
@pytest.mark.parametrize("releaser_first", [False, True])
def test_holders_of_one_page_in_one_compaction(fill, releaser_first):
    """What a sequence may do follows from the pages' holders before the call: slot 1 gives up a
    shared page, slot 2 would move tokens in it and is refused, wherever the two stand in the batch."""
    c = cache(fill + 3, 4, 3 * fill + 10, layers=1)
    c.alloc(ints([1]), ints([32]))
    c.fork(ints([1]), ints([2]))
    rest = list(range(3, fill + 3))
    if rest:
        c.alloc(ints(rest), ints([20 + s % 9 for s in rest]))
    start = [t.clone() for t in (c.page_table, c.lens, c.refs, c.k, c.v)]
    keep = tokens(c, 2)
    jobs = {1: (20, []), 2: (6, [2, 4])}  # (drafted tokens, accepted path)
    jobs.update({s: (10, [1, 3 + s % 6]) for s in rest})
    for at in (0, fill // 2, fill):
        order = list(rest)
        order.insert(at, 1 if releaser_first else 2)
        order.insert(0 if not releaser_first and at else len(order), 2 if releaser_first else 1)
        for t, x in zip((c.page_table, c.lens, c.refs, c.k, c.v), start):
            t.copy_(x)
        path = [list(jobs[s][1]) + [-1] * (2 - len(jobs[s][1])) for s in order]
        c.compact(tree.cu_of([jobs[s][0] for s in order]), ints(path), ints([len(jobs[s][1]) for s in order]), slots=ints(order))
        with pytest.raises(ea.AttnError):
            ea.get_device_status()
        assert c.lens.tolist() == [0, 12, 32] + [20 + s % 9 - 8 for s in rest]
        same(keep, tokens(c, 2))
        assert c.refs[c.page_table[2, 1]] == 1 and c.refs[c.page_table[2, 0]] == 2
        sound(c)


def test_requests_whose_sum_passes_32_bits():
    """Each asks for almost as many pages as a row of the table has entries: none fits, none behind
    them that needs a page, and what needs none is granted."""
    width = (2 ** 31 - 4096) // 16
    n = 40
    table = torch.empty((n + 2, width), dtype=torch.int32, device="cuda")
    table[:, :4] = -1
    kv = torch.zeros(1, 64, 16, 1, 64, dtype=torch.bfloat16, device="cuda")
    zero = torch.zeros(n + 2, dtype=torch.int32, device="cuda")
    c = ea.KVCache(kv, kv.clone(), table, zero, torch.zeros(64, dtype=torch.int32, device="cuda"))
    assert c.alloc(ints([0]), ints([20])).tolist() == [1]
    for m in (n, 32, 17):
        slots = list(range(1, m + 1))
        want = [width * 16 - i % 3 for i in range(m)]
        granted = c.alloc(ints(slots + [0, m + 1]), ints(want + [21, 5])).tolist()
        assert granted == [0] * m + [1, 0]
        assert c.lens.tolist()[:m + 2] == [21] + [0] * (m + 1)
        assert c.page_table[:, :4].tolist() == [[0, 1, -1, -1]] + [[-1] * 4] * (n + 1)
        assert c.refs.tolist() == [1, 1] + [0] * 62
    ea.get_device_status()
