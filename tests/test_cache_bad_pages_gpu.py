"""A page number out of range in a slot's table: the operators leave that sequence alone, do the
others, and report it."""
import pytest
import torch

import exact_attention_103_b200 as ea
import test_tree_gpu as tree

pytestmark = pytest.mark.gpu
ints = tree.ints
BAD = (-1, 10 ** 6, 2 ** 31 - 1, -2 ** 31)


def reported():
    with pytest.raises(ea.AttnError) as e:
        ea.get_device_status()
    assert e.value.status == ea.ATTN_ERR_INVALID_ARG


@pytest.mark.parametrize("dtype,d", tree.KINDS)
@pytest.mark.parametrize("n,G", [(1, 4), (6, 4), (12, 4), (25, 4), (50, 4)])
def test_attention(dtype, d, n, G):
    """Any page of a sequence, in every form, in short items and in ones that many SMs share."""
    ctx = [100, 9000, 300, 64]
    c = tree.build(ctx, [n] * 4, 2, d, 64, dtype, seed=5)
    mask = tree.tree_mask([n] * 4, 7)
    q, cu, o, lse = tree.run(c, [n] * 4, 2 * G, mask)
    keep = c.page_table.clone()
    for i, (b, m) in enumerate([(0, 0), (0, 1), (1, 0), (1, 60), (1, (9000 + n - 1) // 64), (2, 3), (3, 0)]):
        c.page_table[b, m] = BAD[i % 4]
        o2, lse2 = torch.full_like(o, 7.0), torch.full_like(lse, 7.0)
        ea.tree_fwd(c, q, cu, mask=mask, out=o2, lse=lse2)
        reported()
        own = slice(b * n, (b + 1) * n)
        assert (o2[own] == 7).all() and (lse2[:, own] == 7).all()
        o2[own], lse2[:, own] = o[own], lse[:, own]
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        c.page_table.copy_(keep)
    o2, lse2 = ea.tree_fwd(c, q, cu, mask=mask)
    ea.get_device_status()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_attention_of_many_short_sequences():
    """Items far shorter than what the copies run ahead."""
    ctx = [3 + b % 5 for b in range(600)]
    c = tree.build(ctx, [1] * 600, 2, 64, 16, seed=6)
    q, cu, o, lse = tree.run(c, [1] * 600, 4)
    bad = list(range(0, 600, 7))
    c.page_table[bad, 0] = c.pages
    o2, lse2 = torch.full_like(o, 7.0), torch.full_like(lse, 7.0)
    ea.tree_fwd(c, q, cu, out=o2, lse=lse2)
    reported()
    assert (o2[bad] == 7).all() and (lse2[:, bad] == 7).all()
    o2[bad], lse2[:, bad] = o[bad], lse[:, bad]
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_fork():
    c = tree.build([40, 40, 48, 0, 0, 0], [0] * 6, 2, 64, 16, layers=2, spare=4)
    state = [t.clone() for t in (c.page_table, c.lens, c.refs)]
    for slot, m, src, dst in ((0, 0, [0, 1, 2], [3, 4, 5]), (0, 2, [1, 0, 2], [4, 3, 5]), (2, 1, [0, 2, 1], [5, 3, 4])):
        for page in BAD:
            for t, s in zip((c.page_table, c.lens, c.refs), state):
                t.copy_(s)
            c.page_table[slot, m] = page
            before = [t.clone() for t in (c.page_table, c.lens, c.refs)]
            granted = c.fork(ints(src), ints(dst))
            reported()
            assert granted.tolist() == [int(s != slot) for s in src]
            assert c.lens[3] == 0 and (c.page_table[3] == before[0][3]).all()
            for s, t in zip(src, dst):
                if s != slot:
                    full = int(state[1][s]) // 16
                    assert c.lens[t] == state[1][s] and torch.equal(c.page_table[t, :full], c.page_table[s, :full])
            held = torch.zeros_like(c.refs)
            for s in range(6):
                for p in c.page_table[s, :-(-int(c.lens[s]) // 16)].tolist():
                    if 0 <= p < c.pages:
                        held[p] += 1
            # the page that the bad number stands for keeps the count its owner gave it
            lost = before[2] - torch.stack([held, before[2]]).amin(0)
            assert torch.equal(c.refs, held + lost)


def test_compact():
    """The page that a token moves from, or to."""
    for m in (1, 3):  # tokens 16.., 48.. of 10 + 50
        for page in BAD:
            c = tree.build([10, 10], [50, 50], 2, 64, 16, layers=2, seed=7)
            other = tree.build([10, 10], [50, 50], 2, 64, 16, layers=2, seed=7)
            path = ints([[0, 3, 8, 41], [0, 3, 8, 41]])
            c.page_table[0, m] = page
            before = [t.clone() for t in (c.page_table, c.lens, c.refs)]
            # token 10 + 8 (page 1) moves to 12, token 51 (page 3) to 13
            c.compact(ints([0, 50, 100]), path, ints([4, 4]))
            reported()
            other.compact(ints([0, 50]), path[1:], ints([4]), slots=ints([1]))
            for name in ("k", "v"):
                assert torch.equal(getattr(c, name).view(torch.uint8), getattr(other, name).view(torch.uint8))
            assert c.lens.tolist() == [60, 14] and torch.equal(c.page_table[0], before[0][0])
            assert torch.equal(c.page_table[1], other.page_table[1])


def test_compact_along_bad_paths():
    """Path entries that name no token: negative behind negative, far out, falling."""
    c = tree.build([40], [20], 2, 64, 16, layers=2, seed=8, fill=1.0)
    before = [t.clone() for t in (c.page_table, c.lens, c.refs, c.k, c.v)]
    low = -2 ** 31
    for path in ([low, low + 1, low + 2], [-3, -2, -1], [-1, 0, 1], [5, 4, 6], [0, 0, 1], [0, 1, 20], [0, 1, 2 ** 31 - 1], [1, low, 3]):
        c.compact(ints([0, 20]), ints([path]), ints([3]))
        reported()
        assert all(torch.equal(x, y) for x, y in zip(before, (c.page_table, c.lens, c.refs, c.k, c.v)))


def test_append_leaves_the_queries_too():
    """A sequence that cannot be appended: neither its rows of the cache nor its rotated queries."""
    c = tree.build([20, 20, 20], [4, 4, 4], 1, 64, 16, fill=2.0)
    plan = ea.Rope(64)
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn((12, h, 64), generator=g, device="cuda").to(torch.bfloat16) for h in (3, 1, 1))
    cu = ints([0, 4, 8, 12])
    want = ea.rope_append(c, q, k, v, cu, plan=plan)
    ea.get_device_status()
    keep = c.page_table.clone()

    def again(**kw):
        out = torch.full_like(q, 7.0)
        k0, v0 = c.k.clone(), c.v.clone()
        ea.rope_append(c, q, -k, -v, cu, plan=plan, out=out, **kw)
        reported()
        assert (out[4:8] == 7).all() and torch.equal(out[:4], want[:4]) and torch.equal(out[8:], want[8:])
        page = int(keep[1, 1])
        assert torch.equal(c.k[0, page], k0[0, page]) and torch.equal(c.v[0, page], v0[0, page])
    c.page_table[1, 1] = -1
    again()
    c.page_table.copy_(keep)
    again(slots=ints([0, 9, 2]))
    again(slots=ints([0, 0, 2]))
    c.lens[1] = 3
    again()


def test_append_to_one_slot_twice_behind_a_bad_page():
    """The second of two sequences with one slot is refused whatever the pages of its first tokens are."""
    for _ in range(20):
        c = tree.build([10], [20], 2, 64, 16, fill=1.0)
        g = torch.Generator(device="cuda").manual_seed(2)
        x = torch.randn((40, 2, 64), generator=g, device="cuda").to(torch.bfloat16)
        page = int(c.page_table[0, 1])
        c.page_table[0, 0] = c.pages
        ea.rope_append(c, None, x, x, ints([0, 20, 40]), slots=ints([0, 0]))
        reported()
        for t in (c.k, c.v):
            assert torch.equal(t[0, page, :14], x[6:20])
