"""Plain 64-bit references of the serving operators (rotary positions, the paged cache and
attention over it) for the tests: written from the definitions, sharing nothing with the
CUDA path."""
from __future__ import annotations

import math

import torch


def rope_freqs(dim, base=10000.0, scaling=None, factor=1.0, original_len=None, fast=32.0, slow=1.0):
    """(frequencies float64 [dim/2] in radians per position, amplitude)."""
    i = torch.arange(dim // 2, dtype=torch.float64)
    if scaling == "ntk":
        base = base * factor ** (dim / (dim - 2))
    f = base ** (-2 * i / dim)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling != "yarn":
        return f, 1.0

    def at(turns):
        return dim * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(base))
    lo, hi = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), dim // 2 - 1)
    ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return f * (1 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1


def rope(x, pos, freqs, amp, inter, inverse=False):
    """x [..., T, H, d] float64 rotated at pos [..., T]; freqs [dim/2]."""
    dim = 2 * freqs.numel()
    a = pos.double()[..., None, None] * freqs * (-1 if inverse else 1)
    c, s = a.cos() * amp, a.sin() * amp
    y = x.clone()
    u, v = (x[..., 0:dim:2], x[..., 1:dim:2]) if inter else (x[..., :dim // 2], x[..., dim // 2:dim])
    p, q = u * c - v * s, v * c + u * s
    if inter:
        y[..., 0:dim:2], y[..., 1:dim:2] = p, q
    else:
        y[..., :dim // 2], y[..., dim // 2:dim] = p, q
    return y


class Book:
    """Tables of a paged cache kept with Python lists: the definition of its page operations.
    Data: list `data` of tensors [layers, pages, page, ...] moved along."""

    def __init__(self, slots, max_pages, pages, page, data=()):
        self.page, self.max_pages = page, max_pages
        self.table = [[-1] * max_pages for _ in range(slots)]
        self.lens, self.refs, self.data = [0] * slots, [0] * pages, list(data)

    def count(self, n):
        return -(-n // self.page)

    def free_pages(self):
        return [i for i, r in enumerate(self.refs) if r == 0]

    def _cut(self, s, new):
        for m in range(self.count(new), self.count(self.lens[s])):
            self.refs[self.table[s][m]] -= 1
            self.table[s][m] = -1
        self.lens[s] = new

    def _serve(self, needs, valid):
        """Pages for each request in order, or None: (upto <= free) decides."""
        pool, upto, got = self.free_pages(), 0, []
        for need, ok in zip(needs, valid):
            if not ok:
                got.append(None)
                continue
            a, upto = upto, upto + need
            got.append(pool[a:upto] if need == 0 or upto <= len(pool) else None)
        return got

    def alloc(self, slots, want):
        seen, valid = set(), []
        for s, w in zip(slots, want):
            ok = 0 <= s < len(self.lens) and s not in seen
            seen.add(s)
            valid.append(ok and self.lens[s] <= w <= self.max_pages * self.page)
        needs = [self.count(w) - self.count(self.lens[s]) if ok else 0 for s, w, ok in zip(slots, want, valid)]
        told = []
        for s, w, got in zip(slots, want, self._serve(needs, valid)):
            told.append(int(got is not None))
            if got is not None:
                for m, p in enumerate(got, self.count(self.lens[s])):
                    self.table[s][m] = p
                    self.refs[p] = 1
                self.lens[s] = w
        return told

    def free(self, slots):
        for s in slots:
            if 0 <= s < len(self.lens):
                self._cut(s, 0)

    def fork(self, src, dst):
        before = list(self.lens)
        seen, valid = set(), []
        for a, b in zip(src, dst):
            ok = 0 <= b < len(before) and b not in seen
            seen.add(b)
            valid.append(ok and 0 <= a < len(before) and a != b and before[b] == 0)
        needs = [int(ok and before[a] % self.page != 0) for a, ok in zip(src, valid)]
        told = []
        for a, b, got in zip(src, dst, self._serve(needs, valid)):
            told.append(int(got is not None))
            if got is None:
                continue
            n = before[a]
            for m in range(n // self.page):
                self.table[b][m] = self.table[a][m]
                self.refs[self.table[a][m]] += 1
            for p in got:
                self.table[b][n // self.page] = p
                self.refs[p] = 1
                for c in self.data:
                    c[:, p, :n % self.page] = c[:, self.table[a][n // self.page], :n % self.page]
            self.lens[b] = n
        return told

    def compact(self, cu, path, accepted, slots):
        for b, s in enumerate(slots):
            n, keep = cu[b + 1] - cu[b], path[b][:accepted[b]]
            if (s in slots[:b] or not 0 <= s < len(self.lens) or self.lens[s] < n or len(keep) != accepted[b]
                    or any(not 0 <= p < n for p in keep) or any(x >= y for x, y in zip(keep, keep[1:]))):
                continue
            base = self.lens[s] - n
            for i, p in enumerate(keep):
                x, y = base + p, base + i
                for c in self.data:
                    c[:, self.table[s][y // self.page], y % self.page] = \
                        c[:, self.table[s][x // self.page], x % self.page].clone()
            self._cut(s, base + len(keep))


def gather(cache_layer, row, n, page):
    """Tokens 0..n-1 of a table row from one layer [pages, page, heads, d]."""
    idx = torch.tensor(row[:-(-n // page)] if n else [], dtype=torch.long, device=cache_layer.device)
    return cache_layer[idx].flatten(0, 1)[:n]


def attend(q, k, v, seen, scale):
    """q [n, Hq, d], k and v [L, Hkv, d], seen [n, L]: (O, LSE [n, Hq], A = sum p|v|, F), all
    float64; F = sum |v| over the visible keys / sum exp(s - max)."""
    n, Hq, d = q.shape
    G = Hq // k.shape[1]
    q, k, v = q.double(), k.double(), v.double()
    o, a, f = (torch.zeros(n, Hq, d, dtype=torch.float64, device=q.device) for _ in range(3))
    lse = torch.full((n, Hq), float("-inf"), dtype=torch.float64, device=q.device)
    for h in range(Hq):
        kh, vh = k[:, h // G], v[:, h // G]
        s = torch.where(seen, (q[:, h] @ kh.t()) * scale, float("-inf"))
        m = s.amax(-1, keepdim=True) if s.shape[1] else torch.full((n, 1), float("-inf"), device=q.device)
        some = torch.isfinite(m[:, 0])
        if not some.any():
            continue
        e = torch.where(seen, (s - m.nan_to_num(neginf=0.0)).exp(), 0.0)[some]
        l = e.sum(-1, keepdim=True)
        o[some, h], a[some, h] = (e / l) @ vh, (e / l) @ vh.abs()
        f[some, h] = (seen[some].double() @ vh.abs()) / l
        lse[some, h] = (l.log() + m[some])[:, 0]
    return o, lse, a, f
