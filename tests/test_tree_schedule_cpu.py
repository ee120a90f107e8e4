"""A step-by-step twin of the work list of the attention over the paged cache: every key tile of
every (sequence, cache head, row pair) belongs to exactly one CTA, a CTA leaves at most two unfinished
parts, and the parts that the second launch joins are those of one item in the order of its keys.
And the kernel's register split, read from its source."""
import pathlib
import random
import re

import pytest

SOURCE = (pathlib.Path(__file__).parents[1] / "exact_attention_103_b200" / "csrc" / "attn_tree_sm100.cu").read_text()
COSTS = [(4, 7, 20), (2, 4, 10), (2, 4, 20)]  # one row tile, two, beginning an item: bf16 d 128, bf16 d 64, E4M3
MIN_PART = int(re.search(r"constexpr int kMinPart = (\d+);", SOURCE).group(1))


def ceil(a, b):
    return -(-a // b)


class List:
    def __init__(self, n, lens, heads, G, masked, costs):
        self.n, self.lens, self.heads, self.masked = n, lens, heads, masked
        self.tpt, (self.one, self.pair, self.item) = 128 // G, costs
        self.cum = [0]
        for b in range(len(n)):
            work = sum(self.item + self.tiles(b, rt) * self.cost(b, rt) for rt in range(ceil(n[b], 2 * self.tpt)))
            self.cum.append(self.cum[-1] + work * heads)

    def tiles(self, b, rt):
        end = self.n[b] if self.masked else min((rt + 1) * 2 * self.tpt, self.n[b])
        return ceil(self.lens[b] - self.n[b] + end, 128)

    def cost(self, b, rt):
        return self.pair if self.n[b] - rt * 2 * self.tpt > self.tpt else self.one

    def at(self, x, end):
        b = max(i for i in range(len(self.n)) if self.cum[i] <= x and self.cum[i] < self.cum[i + 1])
        per_head = (self.cum[b + 1] - self.cum[b]) // self.heads
        h, r = divmod(x - self.cum[b], per_head)
        rt = 0
        while r >= self.item + self.tiles(b, rt) * self.cost(b, rt):
            r -= self.item + self.tiles(b, rt) * self.cost(b, rt)
            rt += 1
        kv, w = self.tiles(b, rt), self.cost(b, rt)
        begin = x - r
        after = min(end, begin + self.item + kv * w)
        return ((b, h, rt), ceil(max(0, r - self.item), w), ceil(max(0, after - begin - self.item), w), kv, begin,
                after, w)


@pytest.mark.parametrize("seed", range(300))
def test_every_tile_once_and_parts_join(seed):
    r = random.Random(seed)
    B, heads, G, masked = r.randint(1, 6), r.choice([1, 2, 3]), r.choice([1, 3, 4, 8, 128]), r.random() < 0.5
    n = [r.choice([0, 1, r.randint(1, 256), 5 if masked else r.randint(1, 900)]) for _ in range(B)]
    lens = [x + r.choice([0, r.randint(0, 3000)]) for x in n]
    w = List(n, lens, heads, G, masked, COSTS[seed % 3])
    total = w.cum[-1]
    want = {((b, h, rt), j) for b in range(B) for h in range(heads) for rt in range(ceil(n[b], 2 * w.tpt))
            for j in range(w.tiles(b, rt))}
    ctas = max(1, min(r.choice([1, 2, 7, 148]), total // MIN_PART)) if total else 0
    owner, parts, joins = {}, {}, []
    for c in range(ctas):
        x, end = c * total // ctas, (c + 1) * total // ctas
        while x < end:
            item, j0, j1, kv, begin, x, cost = w.at(x, end)
            if j0 >= j1:
                continue
            for j in range(j0, j1):
                assert (item, j) not in owner
                owner[item, j] = c
            if j0 > 0 or j1 < kv:
                slot = (c, 1 if j0 == 0 else 0)
                assert slot not in parts
                parts[slot] = (item, j0, j1, kv)
            if j0 == 0 and j1 < kv:
                at = begin + w.item + (kv - 1) * cost  # the first unit of the item's last tile
                last = at * ctas // total
                while (last + 1) * total // ctas <= at:
                    last += 1
                while last * total // ctas > at:
                    last -= 1
                joins.append((c, last))
    assert set(owner) == want
    joined = set()
    for c, last in joins:
        j = 0
        for k in range(c, last + 1):
            item, j0, j1, kv = parts[k, 1 if k == c else 0]
            assert item == parts[c, 1][0] and j0 == j
            j = j1
            joined.add((k, 1 if k == c else 0))
        assert j == kv
    assert joined == set(parts)


def test_costs_are_the_kernels():
    line = re.search(r"COST_ONE = (.*?), COST_PAIR = (.*?),\s+COST_ITEM = (.*?);", SOURCE, re.S).groups()
    for (f8, d), costs in zip([(False, 128), (False, 64), (True, 128)], COSTS):
        env = {"F8": f8, "D": d}
        got = []
        for e in line:
            m = re.fullmatch(r"(.*?) \? (\d+) : (\d+)", e)
            cond = m.group(1).replace("!F8", "not F8").replace("&&", "and").replace("||", "or")
            got.append(int(m.group(2 if eval(cond, {}, env) else 3)))
        assert tuple(got) == costs
    assert MIN_PART >= max(c[1] for c in COSTS)


def test_register_split():
    inc = int(re.search(r"setmaxnreg\.inc\.sync\.aligned\.u32 (\d+)", SOURCE).group(1))
    dec = int(re.search(r"setmaxnreg\.dec\.sync\.aligned\.u32 (\d+)", SOURCE).group(1))
    threads = int(re.search(r"constexpr int kThreads = (\d+);", SOURCE).group(1))
    launch = 65536 // threads // 8 * 8  # registers a thread at launch, one CTA per SM
    assert SOURCE.count("setmaxnreg") == 2 and inc % 8 == 0 and dec % 8 == 0
    assert 256 * inc + (threads - 256) * dec <= threads * launch
