"""Random histories of a cache whose slots share pages freely (drafted tokens may lie in pages that a
fork holds too) against the same operations on Python lists: tables, lengths, counts and every byte."""
import random

import pytest
import torch

import exact_attention_103_b200 as ea
import serve_ref as ref
import test_cache_pages_gpu as pages

pytestmark = pytest.mark.gpu


class Book(ref.Book):
    """With the rules for shared pages: growth inside one takes a page of its own first, and compaction
    moves nothing in one; both by the counts before the call."""

    def alloc(self, slots, want):
        seen, valid, alone = set(), [], []
        for s, w in zip(slots, want):
            ok = s not in seen and self.lens[s] <= w <= self.max_pages * self.page
            seen.add(s)
            valid.append(ok)
            n = self.lens[s]
            alone.append(ok and w > n and n % self.page != 0 and self.refs[self.table[s][n // self.page]] > 1)
        needs = [self.count(w) - self.count(self.lens[s]) + a if ok else 0
                 for s, w, ok, a in zip(slots, want, valid, alone)]
        told = []
        for s, w, a, got in zip(slots, want, alone, self._serve(needs, valid)):
            told.append(int(got is not None))
            if got is None:
                continue
            n = self.lens[s]
            for m, p in enumerate(got, n // self.page if a else self.count(n)):
                if a and m == n // self.page:
                    old = self.table[s][m]
                    self.refs[old] -= 1
                    for c in self.data:
                        c[:, p, :n % self.page] = c[:, old, :n % self.page]
                self.table[s][m] = p
                self.refs[p] = 1
            self.lens[s] = w
        return told

    def compact(self, cu, path, accepted, slots):
        refs, fine = list(self.refs), []
        for b, s in enumerate(slots):
            base = self.lens[s] - (cu[b + 1] - cu[b])
            fine.append(all(p == i or refs[self.table[s][(base + i) // self.page]] == 1
                            for i, p in enumerate(path[b][:accepted[b]])))
        for b, s in enumerate(slots):
            if fine[b]:
                super().compact([0, cu[b + 1] - cu[b]], [path[b]], [accepted[b]], [s])
        return all(fine)


@pytest.mark.parametrize("seed,page,layers,heads,d,dtype", [
    (1, 16, 1, 1, 64, torch.bfloat16), (2, 16, 3, 3, 64, torch.float8_e4m3fn), (3, 32, 2, 2, 128, torch.bfloat16),
    (4, 16, 2, 1, 128, torch.bfloat16), (5, 64, 1, 2, 64, torch.float8_e4m3fn)])
def test_histories(seed, page, layers, heads, d, dtype):
    r = random.Random(seed)
    n_slots = 24
    p = pages.Pair(n_slots, 5, 60, page, layers, heads, d, dtype, seed)
    p.b = Book(n_slots, 5, 60, page, p.b.data)
    copied = 0
    for step in range(150):
        kind = r.choice(["alloc", "alloc", "free", "fork", "compact", "compact"])
        empty = [s for s in range(n_slots) if p.b.lens[s] == 0]
        held = [s for s in range(n_slots) if p.b.lens[s] > 0]
        good = True
        if kind == "alloc":
            slots = r.sample(range(n_slots), r.randint(1, 10))
            before = [x for row in p.b.table for x in row]
            p.alloc(slots, [min(5 * page, p.b.lens[s] + r.randint(0, 2 * page)) for s in slots])
            copied += sum(x >= 0 and x != y for x, y in zip(before, [x for row in p.b.table for x in row]))
        elif kind == "free" and held:
            p.free(r.sample(held, r.randint(1, min(3, len(held)))))
        elif kind == "fork" and held and empty:
            n = r.randint(1, min(8, len(empty)))
            p.fork([r.choice(held) for _ in range(n)], r.sample(empty, n))
        elif kind == "compact" and held:
            slots = r.sample(held, r.randint(1, min(8, len(held))))
            drafted = [r.randint(0, min(p.b.lens[s], 2 * page)) for s in slots]
            path = [list(range(r.randint(0, n))) if r.random() < 0.5 else sorted(r.sample(range(n), r.randint(0, n)))
                    for n in drafted]
            cu = [sum(drafted[:i]) for i in range(len(drafted) + 1)]
            width = max([1] + [len(x) for x in path])
            grid = [x + [-1] * (width - len(x)) for x in path]
            took = [len(x) for x in path]
            p.c.compact(pages.ints(cu), pages.ints(grid), pages.ints(took), slots=pages.ints(slots))
            good = p.b.compact(cu, grid, took, slots)
        p.same()
        if good:
            ea.get_device_status()
        else:
            with pytest.raises(ea.AttnError):
                ea.get_device_status()
    assert copied > 0
