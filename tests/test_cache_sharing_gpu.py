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
