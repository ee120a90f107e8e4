"""Cases and plain forms of the serving operators: rotary positions (with their gradient and
their cache-writing form), attention of drafted tokens over a paged cache, and the
management of the cache's pages.

``run`` computes an operator in elementary torch operations (``own`` false) or calls the
framework's operator (``own`` true); ``exact`` computes the same from the definitions in
64 bits, sequence by sequence.  A case fixes every shape, sequence length and tree; the seed
gives the values, and which pages of the cache a sequence owns.

The cache: K and V are ``[layers, pages, page, heads, d]``; row s of ``table`` lists the pages
of sequence slot s (-1 behind its last), ``lens`` its tokens, ``refs`` how many slots hold a
page (0: free).  Drafted tokens are the last tokens of their sequence in the cache.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
         "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}
# the two scales of an E4M3 cache: stored value * scale = real value
K_SCALE, V_SCALE = 0.0625, 0.03125
YARN = dict(scaling="yarn", factor=8.0, original_len=4096)


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # a training prompt, dense: the shape of the repository's causal benchmark workload
        dict(name="rope prefill", op="rope", dir="fwd", dtype="bf16", B=2, lo=8192, hi=8192, Hq=16,
             Hk=16, d=128, rot=128, inter=False, scaling="none", packed=False, pick=1),
        # gradients of a packed batch (16 sequences of 512 to 16384 tokens), half of each head
        # rotated, pairs interleaved, positions scaled for a context beyond the trained one
        dict(name="rope gradient packed", op="rope", dir="bwd", dtype="bf16", B=16, lo=512, hi=16384,
             Hq=16, Hk=16, d=128, rot=64, inter=True, scaling="yarn", packed=True, pick=1),
        # one serving step of a batch: a token each
        dict(name="append single tokens", op="append", B=48, n=1, Hq=32, Hkv=8, d=128, page=16, lo=200,
             hi=1000, cache="bf16", rot=128, inter=False, pick=2),
        # drafted trees written into an 8-bit cache
        dict(name="append trees e4m3", op="append", B=32, n=61, Hq=32, Hkv=8, d=128, page=64, lo=100,
             hi=2000, cache="e4m3", rot=64, inter=True, pick=3),
        # one user, a short context, no grouped heads: latency counts
        dict(name="attend one short", op="tree", B=1, n=1, Hq=16, Hkv=16, d=128, page=16, lo=1003,
             hi=1003, cache="bf16", mask="chain", pick=4),
        # a serving batch of single tokens over ragged contexts
        dict(name="attend batch", op="tree", B=64, n=1, Hq=32, Hkv=8, d=128, page=64, lo=512, hi=8192,
             cache="bf16", mask="chain", pick=5),
        # verification of drafted trees, ragged sizes
        dict(name="attend trees", op="tree", B=16, n=48, Hq=32, Hkv=8, d=128, page=32, lo=1000,
             hi=16384, cache="bf16", mask="tree", pick=6),
        # two very long contexts in an 8-bit cache
        dict(name="attend long e4m3", op="tree", B=2, n=16, Hq=32, Hkv=8, d=128, page=128, lo=120000,
             hi=131072, cache="e4m3", mask="tree", pick=7),
        # a chunk of a prompt behind what is cached already
        dict(name="attend chunk d64", op="tree", B=4, n=700, Hq=16, Hkv=16, d=64, page=16, lo=1, hi=4096,
             cache="bf16", mask="chain", pick=8),
        # search over several continuations: old branches dropped, kept ones forked
        dict(name="fork", op="fork", B=48, slots=256, layers=8, pages=4096, page=16, Hkv=8, d=128,
             lo=17, hi=900, pick=9),
        # after verification: the accepted path moved together, surplus pages released
        dict(name="compact", op="compact", B=64, slots=80, layers=8, pages=2500, page=16, Hkv=8, d=128,
             lo=20, hi=500, n=48, accept=8, pick=10),
        # sequences retire and others are admitted, a large pool
        dict(name="retire and admit", op="pages", B=128, slots=1024, pages=65536, page=16, lo=1,
             hi=900, pick=11),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    pick = rng.randrange(1 << 20)
    op = rng.choice(["rope", "append", "tree", "tree", "tree", "fork", "compact", "pages", "copy"])
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 8, 16])
    G = rng.choice([1, 2, 4, 4, 7, 8])
    if op == "rope":
        B = _log(rng, 1, 16)
        Hq, Hk = min(Hkv * G, 32), Hkv
        hi = _log(rng, 1, min(8192, 200000000 // (B * (Hq + Hk) * d)))
        packed = rng.random() < 0.5
        return dict(op=op, dir=rng.choice(["fwd", "bwd"]), dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    B=B, lo=max(1, hi // 4) if packed else hi, hi=hi, Hq=Hq, Hk=Hk, d=d,
                    rot=rng.choice([d, d // 2, d // 4]), inter=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]), packed=packed, pick=pick)
    if op == "append":
        hi = _log(rng, 2, 2000)
        return dict(op=op, B=_log(rng, 1, 64), n=_log(rng, 1, 100), Hq=Hkv * G, Hkv=Hkv, d=d, page=page,
                    lo=max(1, hi // 3), hi=hi, cache=rng.choice(["bf16", "e4m3"]),
                    rot=rng.choice([d, d // 2]), inter=rng.random() < 0.5, pick=pick)
    if op == "tree":
        mask = rng.choice(["chain", "tree"])
        n = rng.choice([1, _log(rng, 2, 128), _log(rng, 2, 600 if mask == "chain" else 256)])
        cache = rng.choice(["bf16", "e4m3"])
        # the tokens of all sequences together stay within the listed cases' cost
        most = min(131072, 262144 * 8 // (max(Hkv, 4) * max(1, n * G // 64)))
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, max(2, most // B))
        return dict(op=op, B=B, n=n, Hq=Hkv * G, Hkv=Hkv, d=d, page=page, lo=max(1, hi // rng.choice([1, 4, 50])),
                    hi=hi, cache=cache, mask=mask, pick=pick)
    hi = _log(rng, 2, 600)
    lo = max(1, hi // 8)
    layers = rng.randint(1, 8)
    B = _log(rng, 1, 64)
    Hkv = min(Hkv, 8)
    if op == "pages":
        slots = B + _log(rng, 1, 900)
        return dict(op=op, B=B, slots=slots, pages=max(1024, slots * (hi // page + 1) + _log(rng, 1, 9000)),
                    page=page, lo=lo, hi=hi, pick=pick)
    if op == "copy":
        pages = _log(rng, 64, 131072 // (page * 2))
        return dict(op=op, B=max(1, pages // rng.choice([3, 5, 20])), layers=layers, pages=pages, page=page,
                    Hkv=Hkv, d=d, pick=pick)
    n = _log(rng, 2, 128)
    per = (hi + (n if op == "compact" else 0)) // page + 2
    B = min(B, max(1, 65536 // (page * 2 * per)))
    slots = 2 * B + rng.randint(0, 9) if op == "fork" else B + rng.randint(0, 9)
    case = dict(op=op, B=B, slots=slots, layers=layers, pages=2 * B * per + rng.randint(8, 90), page=page, Hkv=Hkv,
                d=d, lo=lo, hi=hi, pick=pick)
    if op == "compact":
        case.update(n=n, accept=rng.randint(1, min(n, 12)))
    return case


def _lengths(case):
    """Contexts of the case's sequences: log-uniform over [lo, hi], the longest among them."""
    r = random.Random(case["pick"])
    lo, hi = case["lo"], case["hi"]
    got = [_log(r, lo, hi) for _ in range(case["B"])]
    got[r.randrange(len(got))] = hi
    return [min(max(g, lo), hi) for g in got]


def _drafted(case):
    """Drafted tokens of each sequence: n, or with a tree of several sequences n/2 to n."""
    r = random.Random(case["pick"] + 1)
    n, B = case["n"], case["B"]
    if case.get("mask") == "chain" and n <= 128 or n == 1:
        return [n] * B
    return [n] + [r.randint((n + 1) // 2, n) for _ in range(B - 1)]


def _trees(case, drafted):
    """(depth [T], visible [T, W]) of random trees: a node sees itself and its ancestors."""
    r = random.Random(case["pick"] + 2)
    W = max(drafted)
    depth, rows = [], []
    for n in drafted:
        seen = np.zeros((n, W), dtype=bool)
        dep = [0] * n
        for i in range(n):
            parent = r.randint(max(-1, i - 6), i - 1) if i else -1
            if parent >= 0:
                seen[i] = seen[parent]
                dep[i] = dep[parent] + 1
            seen[i, i] = True
        depth += dep
        rows.append(seen)
    return np.array(depth, dtype=np.int32), np.concatenate(rows)


def work(case):
    op = case["op"]
    if op == "rope":
        T = sum(_lengths(case)) if case["packed"] else case["B"] * case["hi"]
        row = (case["Hq"] + case["Hk"]) * case["d"]
        return dict(bytes=2 * T * row * BYTES[case["dtype"]],
                    flops=3 * T * (case["Hq"] + case["Hk"]) * case["rot"])
    if op == "append":
        T, d = sum(_drafted(case)), case["d"]
        return dict(bytes=T * d * (4 * case["Hq"] + 2 * case["Hkv"] * (2 + BYTES[case["cache"]])),
                    flops=3 * T * (case["Hq"] + case["Hkv"]) * case["rot"])
    if op == "tree":
        ctx, drafted, d = _lengths(case), _drafted(case), case["d"]
        if case["mask"] == "tree":
            inside = int(_trees(case, drafted)[1].sum())
        else:
            inside = sum(n * (n + 1) // 2 for n in drafted)
        pairs = inside + sum(n * c for n, c in zip(drafted, ctx))
        T = sum(drafted)
        return dict(bytes=2 * sum(n + c for n, c in zip(drafted, ctx)) * case["Hkv"] * d * BYTES[case["cache"]]
                    + T * case["Hq"] * (4 * d + 4), flops=4 * case["Hq"] * d * pairs)
    if op == "copy":
        return dict(bytes=4 * case["B"] * case["layers"] * case["page"] * case["Hkv"] * case["d"] * 2, flops=0)
    if op == "pages":
        used = sum(-(-c // case["page"]) for c in _lengths(case))
        return dict(bytes=4 * case["pages"] + 16 * used, flops=0)
    row = case["layers"] * case["Hkv"] * case["d"] * 2 * 4  # read and written, K and V
    if op == "fork":
        ctx = _lengths(case)
        return dict(bytes=row * sum(c % case["page"] for c in ctx)
                    + 16 * sum(-(-c // case["page"]) for c in ctx), flops=0)
    _, path, took = _paths(case, _drafted(case))
    moved = sum(int((path[b, :a] != np.arange(a)).sum()) for b, a in enumerate(took))
    return dict(bytes=row * moved + 64 * case["B"], flops=0)


def _paths(case, drafted):
    """Accepted nodes of each tree: (B, most accepted), increasing, -1 behind the last."""
    r = random.Random(case["pick"] + 3)
    took = [r.randint(0, min(case["accept"], n)) for n in drafted]
    path = np.full((len(drafted), max(max(took), 1)), -1, dtype=np.int32)
    for b, (n, a) in enumerate(zip(drafted, took)):
        path[b, :a] = sorted(r.sample(range(n), a))
    return drafted, path, np.array(took, dtype=np.int32)


# ------------------------------------------------------------------------------ inputs
def _ints(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


def _cu(lengths):
    return _ints(np.concatenate([[0], np.cumsum(lengths)]))


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _pool(g, shape, cache):
    """K or V of a cache: normal values, an E4M3 one stored over its scale."""
    x = torch.empty(shape, dtype=TYPES[cache], device=DEV)
    flat = x.view(-1)
    for a in range(0, flat.numel(), 1 << 28):
        m = min(1 << 28, flat.numel() - a)
        flat[a:a + m] = _normal(g, (m,), torch.float32, 16.0 if cache == "e4m3" else 1.0).to(x.dtype)
    return x


def _hold(g, pages, page, slots, counts, table_width):
    """A page table in which slot s owns pages for counts[s] tokens, at places drawn from g."""
    used = -(-torch.tensor(counts, dtype=torch.int64, device=DEV) // page)
    order = torch.randperm(pages, generator=g, device=DEV)
    m = torch.arange(table_width, device=DEV)
    start = torch.cumsum(used, 0) - used
    mine = m[None, :] < used[:, None]
    at = (start[:, None] + m[None, :]).clamp(max=pages - 1)
    table = torch.where(mine, order[at], -1).to(torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    refs.index_add_(0, order[at].reshape(-1), mine.reshape(-1).to(torch.int32))
    return table.contiguous(), _ints(counts), refs


def _scaled(case_scaling):
    return {"none": {}, "linear": dict(scaling="linear", factor=4.0), "ntk": dict(scaling="ntk", factor=4.0),
            "yarn": YARN}[case_scaling]


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "rope":
        dt = TYPES[case["dtype"]]
        lens = _lengths(case) if case["packed"] else [case["hi"]] * case["B"]
        lead = (sum(lens),) if case["packed"] else (case["B"], case["hi"])
        Hq, Hk, d = case["Hq"], case["Hk"], case["d"]
        # q and k are slices of one projection's output, as a model's layer has them
        both = _normal(g, (*lead, Hq + Hk, d), dt)
        s["q"], s["k"] = both[..., :Hq, :], both[..., Hq:, :]
        s["cu"] = _cu(lens) if case["packed"] else None
        # the position of every token, as a plain form needs it
        s["positions"] = torch.cat([torch.arange(n, device=DEV) for n in lens])
        if own:
            import exact_attention_103_b200 as ea
            s["plan"] = ea.Rope(case["rot"], interleaved=case["inter"], device=DEV, **_scaled(case["scaling"]))
        return s
    page = case["page"]
    if op in ("append", "tree"):
        ctx, drafted = _lengths(case), _drafted(case)
        total = [c + n for c, n in zip(ctx, drafted)]
        width = max(-(-t // page) for t in total)
        pages = sum(-(-t // page) for t in total) + 3
        Hq, Hkv, d, T = case["Hq"], case["Hkv"], case["d"], sum(drafted)
        s["table"], s["lens"], s["refs"] = _hold(g, pages, page, case["B"], total, width)
        s["kc"] = _pool(g, (1, pages, page, Hkv, d), case["cache"])
        s["vc"] = _pool(g, (1, pages, page, Hkv, d), case["cache"])
        s["cu"] = _cu(drafted)
        s["seq"] = torch.repeat_interleave(torch.arange(case["B"], device=DEV), torch.tensor(drafted, device=DEV))
        s["q"] = _normal(g, (T, Hq, d), torch.bfloat16)
        if op == "append":
            both = _normal(g, (T, 2 * Hkv, d), torch.bfloat16)
            s["k"], s["v"] = both[:, :Hkv], both[:, Hkv:]
            depth, _ = _trees(case, drafted)
            s["positions"] = _ints(depth) + _ints(ctx)[s["seq"]]
        elif case["mask"] == "tree":
            s["mask"] = torch.from_numpy(_trees(case, drafted)[1]).to(DEV)
        else:
            s["mask"] = None
        if own:
            import exact_attention_103_b200 as ea
            e = case["cache"] == "e4m3"
            s["cache"] = ea.KVCache(s["kc"], s["vc"], s["table"], s["lens"], s["refs"],
                                    k_scale=K_SCALE if e else 1.0, v_scale=V_SCALE if e else 1.0)
            if op == "append":
                s["plan"] = ea.Rope(case["rot"], interleaved=case["inter"], device=DEV)
        return s
    pages = case["pages"]
    if op == "copy":
        shape = (case["layers"], pages, page, case["Hkv"], case["d"])
        s["kc"], s["vc"] = _pool(g, shape, "bf16"), _pool(g, shape, "bf16")
        order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        s["src"], s["dst"] = order[:case["B"]].contiguous(), order[pages - case["B"]:].contiguous()
        s["table"], s["lens"], s["refs"] = _hold(g, pages, page, 1, [0], 1)
    else:
        slots, B = case["slots"], case["B"]
        ctx = _lengths(case)
        r = random.Random(case["pick"] + 4)
        where = r.sample(range(slots), 2 * B if op == "fork" else B)
        counts = [0] * slots
        if op == "pages":  # the other slots hold sequences too, as far as the pool has room
            for i in range(slots):
                counts[i] = _log(r, case["lo"], case["hi"])
            for i, c in zip(where, ctx):
                counts[i] = c
        elif op == "fork":  # the first half is forked into the second, which holds old branches
            for i, c in enumerate(ctx):
                counts[where[i]] = c
                counts[where[B + i]] = 1 + c // 2
        else:
            for i, (c, n) in enumerate(zip(ctx, _drafted(case))):
                counts[where[i]] = c
        width = -(-(case["hi"] + case.get("n", 0)) // page)
        s["table"], s["lens"], s["refs"] = _hold(g, pages, page, slots, counts, width)
        s["slots"] = _ints(where[:B])
        if op == "pages":
            s["want"] = _ints(ctx)
            layers, Hkv, d = 1, 1, 64  # no values move: the smallest cache
            s["kc"] = torch.zeros((layers, pages, page, Hkv, d), dtype=torch.bfloat16, device=DEV)
            s["vc"] = torch.zeros_like(s["kc"])
        else:
            shape = (case["layers"], pages, page, case["Hkv"], case["d"])
            s["kc"], s["vc"] = _pool(g, shape, "bf16"), _pool(g, shape, "bf16")
        if op == "fork":
            s["dst"] = _ints(where[B:])
        if op == "compact":
            drafted, path, took = _paths(case, _drafted(case))
            s["cu"], s["path"], s["took"] = _cu(drafted), _ints(path), _ints(took)
            s["want"] = _ints([c + n for c, n in zip(ctx, drafted)])
    if own:
        import exact_attention_103_b200 as ea
        s["cache"] = ea.KVCache(s["kc"], s["vc"], s["table"], s["lens"], s["refs"])
    return s


# ------------------------------------------------------------------------ plain forms
def _angles(positions, rot, scaling):
    """cos, sin [T, rot/2] in 32 bits of angles taken in 64, and the scaling's amplitude."""
    i = torch.arange(rot // 2, device=DEV, dtype=torch.float64)
    base, amp = 10000.0, 1.0
    if scaling == "ntk":
        base = base * 4.0 ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        f = f / 4.0
    if scaling == "yarn":
        turns = YARN["original_len"] * f / (2 * math.pi)
        # by parts: frequencies of more than 32 turns stay, of less than 1 are divided, a ramp
        # over the index between
        at = [rot * math.log(YARN["original_len"] / (b * 2 * math.pi)) / (2 * math.log(base)) for b in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot // 2 - 1)
        keep = 1 - ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = f * keep + f / YARN["factor"] * (1 - keep)
        amp = 0.1 * math.log(YARN["factor"]) + 1
    a = positions.double()[:, None] * f
    return (a.cos() * amp).float(), (a.sin() * amp).float()


def _rotate(x, cos, sin, rot, inter):
    """x [T, H, d] with its first rot dimensions rotated, in 32 bits."""
    x = x.float()
    r, rest = x[..., :rot], x[..., rot:]
    c, s = cos[:, None], sin[:, None]
    if inter:
        a, b = r[..., 0::2], r[..., 1::2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([y, rest], -1)


def _rows(s, page, at, slots):
    """Cache rows (page * size + offset) of token positions `at` of `slots` (same shape)."""
    at = at.long()
    return s["table"][slots, at // page].long() * page + at % page


def _free(s, page, slots):
    m = torch.arange(s["table"].shape[1], device=DEV)
    held = m[None] < -(-s["lens"][slots] // page)[:, None]
    s["refs"].index_add_(0, s["table"][slots].clamp(min=0).reshape(-1), -held.int().reshape(-1))
    s["table"][slots] = -1
    s["lens"][slots] = 0


def _grant(s, need):
    """The lowest free pages go to `need` in order: (granted, first rank of each, rank of a page)."""
    rank = torch.cumsum((s["refs"] == 0).int(), 0)
    upto = torch.cumsum(need, 0)
    return (need == 0) | (upto <= rank[-1]), upto - need, rank


def _alloc(s, page, slots, want):
    have, new = -(-s["lens"][slots] // page), -(-want // page)
    granted, first, rank = _grant(s, new - have)
    m = torch.arange(s["table"].shape[1], device=DEV)[None]
    take = (m >= have[:, None]) & (m < new[:, None]) & granted[:, None]
    found = torch.searchsorted(rank, (first[:, None] + m - have[:, None] + 1).clamp(min=1))
    found = found.clamp(max=rank.numel() - 1).int()
    s["table"][slots] = torch.where(take, found, s["table"][slots])
    s["refs"].index_add_(0, found.reshape(-1), take.int().reshape(-1))
    s["lens"][slots] = torch.where(granted, want, s["lens"][slots])
    return granted


def _flat(c):
    return c.view(c.shape[0], c.shape[1] * c.shape[2], -1)


def _run_plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "rope":
        cos, sin = _angles(s["positions"], case["rot"], case["scaling"])
        if case["dir"] == "bwd":
            sin = -sin
        out = []
        for x in (s["q"], s["k"]):
            y = _rotate(x.reshape(-1, *x.shape[-2:]), cos, sin, case["rot"], case["inter"])
            out.append(y.to(x.dtype).view(x.shape))
        return out
    page = case["page"]
    if op == "append":
        cos, sin = _angles(s["positions"], case["rot"], "none")
        q = _rotate(s["q"], cos, sin, case["rot"], case["inter"]).to(torch.bfloat16)
        k = _rotate(s["k"], cos, sin, case["rot"], case["inter"])
        v = s["v"].float()
        if case["cache"] == "e4m3":
            k, v = (k / K_SCALE).clamp(-448, 448), (v / V_SCALE).clamp(-448, 448)
        cu, seq = s["cu"].long(), s["seq"]
        local = torch.arange(q.shape[0], device=DEV) - cu[seq]
        rows = _rows(s, page, s["lens"][seq] - (cu[seq + 1] - cu[seq]) + local, seq)
        _flat(s["kc"])[0][rows] = k.flatten(1).to(s["kc"].dtype)
        _flat(s["vc"])[0][rows] = v.flatten(1).to(s["vc"].dtype)
        return q, s["kc"], s["vc"]
    if op == "tree":
        T, Hq, d = s["q"].shape
        B, Hkv, W = case["B"], case["Hkv"], case["n"]
        M = s["table"].shape[1]
        e = case["cache"] == "e4m3"
        pages = s["table"].clamp(min=0).long()
        k, v = (c[0][pages].float().view(B, M * page, Hkv, d) for c in (s["kc"], s["vc"]))
        if e:
            k, v = k * K_SCALE, v * V_SCALE
        cu, seq = s["cu"].long(), s["seq"]
        local = torch.arange(T, device=DEV) - cu[seq]
        n = (cu[1:] - cu[:-1])[:, None, None]
        ctx = s["lens"].long()[:, None, None] - n
        q = torch.zeros((B, W, Hq, d), device=DEV)
        q[seq, local] = s["q"].float()
        j = torch.arange(M * page, device=DEV)[None, None] - ctx  # key as a drafted token
        t = torch.arange(W, device=DEV)[None, :, None]
        if s["mask"] is None:
            seen = (j <= t) & (j < n)
        else:
            full = torch.zeros((B, W, W), dtype=torch.bool, device=DEV)
            full[seq, local, :s["mask"].shape[1]] = s["mask"]
            inside = torch.gather(full, 2, j.clamp(0, W - 1).expand(B, W, -1))
            seen = (j < 0) | (inside & (j < n))
        q = q.view(B, W, Hkv, Hq // Hkv, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, d)
        x = torch.matmul(q, k.permute(0, 2, 3, 1)).view(B, Hkv, W, Hq // Hkv, -1) / math.sqrt(d)
        x = x.masked_fill(~seen[:, None, :, None], float("-inf"))
        top = x.amax(-1, keepdim=True).clamp(min=-1e30)
        p = (x - top).exp()
        total = p.sum(-1, keepdim=True)
        lse = (total.log() + top)[..., 0]
        # values behind a sequence's end count for nothing, whatever the page holds there
        v = v.masked_fill((j[:, 0] >= n[:, 0])[:, :, None, None], 0.0)
        o = torch.matmul((p / total).view(B, Hkv, -1, M * page), v.permute(0, 2, 1, 3))
        o = o.view(B, Hkv, W, Hq // Hkv, d).permute(0, 2, 1, 3, 4).reshape(B, W, Hq, d)
        lse = lse.permute(0, 2, 1, 3).reshape(B, W, Hq)
        return o[seq, local].to(torch.bfloat16), lse[seq, local].t().contiguous()
    if op == "copy":
        src, dst = s["src"].long(), s["dst"].long()
        s["kc"][:, dst] = s["kc"][:, src]
        s["vc"][:, dst] = s["vc"][:, src]
        return s["kc"], s["vc"]
    slots = s["slots"].long()
    if op == "pages":
        _free(s, page, slots)
        granted = _alloc(s, page, slots, s["want"])
        return granted.int(), s["table"], s["lens"], s["refs"]
    if op == "fork":
        dst = s["dst"].long()
        _free(s, page, dst)
        lens, rows = s["lens"][slots], s["table"][slots]
        part = lens % page
        granted, first, rank = _grant(s, (part > 0).int())
        fresh = torch.searchsorted(rank, first + 1).clamp(max=rank.numel() - 1).int()
        m = torch.arange(rows.shape[1], device=DEV)[None]
        whole = (m < (lens // page)[:, None]) & granted[:, None]
        tail = (m == (lens // page)[:, None]) & (granted & (part > 0))[:, None]
        s["table"][dst] = torch.where(whole, rows, torch.where(tail, fresh[:, None], -1))
        s["refs"].index_add_(0, rows.clamp(min=0).reshape(-1), whole.int().reshape(-1))
        s["refs"].index_add_(0, fresh, (granted & (part > 0)).int())
        s["lens"][dst] = torch.where(granted, lens, 0)
        # the copied rows: where there is nothing to copy, a row of the first page onto itself
        old = rows.gather(1, torch.where(part > 0, lens // page, 0).long()[:, None])
        off = torch.arange(page, device=DEV)[None]
        frm = old.long() * page + off
        to = torch.where((off < part[:, None]) & granted[:, None], fresh.long()[:, None] * page + off, frm)
        for c in (_flat(s["kc"]), _flat(s["vc"])):
            c[:, to.reshape(-1)] = c[:, frm.reshape(-1)]
        return granted.int(), s["table"], s["lens"], s["refs"], s["kc"], s["vc"]
    # compact: pages for the drafted tokens, then the accepted path moved together
    _alloc(s, page, slots, s["want"])
    cu, took = s["cu"], s["took"]
    base = s["lens"][slots] - (cu[1:] - cu[:-1])
    i = torch.arange(s["path"].shape[1], device=DEV)[None]
    live = i < took[:, None]
    to = _rows(s, page, base[:, None] + i, slots[:, None])
    frm = torch.where(live, _rows(s, page, base[:, None] + s["path"].clamp(min=0), slots[:, None]), to)
    for c in (_flat(s["kc"]), _flat(s["vc"])):
        c[:, to.reshape(-1)] = c[:, frm.reshape(-1)]
    have, new = -(-s["lens"][slots] // page), -(-(base + took) // page)
    m = torch.arange(s["table"].shape[1], device=DEV)[None]
    drop = (m >= new[:, None]) & (m < have[:, None])
    rows = s["table"][slots]
    s["refs"].index_add_(0, rows.clamp(min=0).reshape(-1), -drop.int().reshape(-1))
    s["table"][slots] = torch.where(drop, -1, rows)
    s["lens"][slots] = base + took
    return s["table"], s["lens"], s["refs"], s["kc"], s["vc"]


# --------------------------------------------------------------- the framework's calls
def _run_own(s):
    import exact_attention_103_b200 as ea
    op = s["case"]["op"]
    if op == "rope":
        f = ea.rope_fwd if s["case"]["dir"] == "fwd" else ea.rope_bwd
        return f(s["plan"], s["q"], s["k"], cu_seqlens=s["cu"])
    c = s["cache"]
    if op == "append":
        q = ea.rope_append(c, s["q"], s["k"], s["v"], s["cu"], plan=s["plan"], positions=s["positions"])
        return q, c.k, c.v
    if op == "tree":
        return ea.tree_fwd(c, s["q"], s["cu"], mask=s["mask"])
    if op == "copy":
        c.copy(s["src"], s["dst"])
        return c.k, c.v
    if op == "pages":
        c.free(s["slots"])
        granted = c.alloc(s["slots"], s["want"])
        return granted, c.page_table, c.lens, c.refs
    if op == "fork":
        c.free(s["dst"])
        granted = c.fork(s["slots"], s["dst"])
        return granted, c.page_table, c.lens, c.refs, c.k, c.v
    c.alloc(s["slots"], s["want"])
    c.compact(s["cu"], s["path"], s["took"], slots=s["slots"])
    return c.page_table, c.lens, c.refs, c.k, c.v


def run(s):
    if own:
        return _run_own(s)
    return _run_plain(s)


# -------------------------------------------------------------------------- in 64 bits
def _turned(x, pos, rot, inter, scaling="none", back=False):
    """x [T, H, d] as complex pairs times e^(i angle), in 64 bits, from the definition."""
    T, H, d = x.shape
    x = x.double()
    base, factor, amp = 10000.0, [1.0] * (rot // 2), 1.0
    if scaling == "linear":
        factor = [4.0] * (rot // 2)
    elif scaling == "ntk":
        base *= 4.0 ** (rot / (rot - 2.0))
    elif scaling == "yarn":
        amp = 1 + 0.1 * math.log(8.0)

        def index_of(turns):  # the (fractional) frequency index that makes `turns` turns over the trained length
            return rot * math.log(4096 / (2 * math.pi * turns)) / (2 * math.log(base))
        lo, hi = max(math.floor(index_of(32)), 0), min(math.ceil(index_of(1)), rot // 2 - 1)
        for i in range(rot // 2):
            ramp = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            factor[i] = 1 / ((1 - ramp) + ramp / 8.0)
    freq = torch.tensor([base ** (-2.0 * i / rot) / factor[i] for i in range(rot // 2)], dtype=torch.float64, device=DEV)
    angle = torch.outer(pos.double(), freq) * (-1 if back else 1)
    spin = torch.polar(torch.full_like(angle, amp), angle)[:, None]
    r = x[..., :rot].reshape(T, H, rot // 2, 2) if inter else x[..., :rot].reshape(T, H, 2, rot // 2).transpose(2, 3)
    y = torch.view_as_real(torch.view_as_complex(r.contiguous()) * spin)
    y = y.reshape(T, H, rot) if inter else y.transpose(2, 3).reshape(T, H, rot)
    return torch.cat([y, x[..., rot:]], 2)


class _Book:
    """The cache's pages kept with Python lists: the definition of alloc, free, fork and compact."""

    def __init__(self, s, page):
        self.page = page
        self.table, self.lens, self.refs = (s[k].cpu().tolist() for k in ("table", "lens", "refs"))

    def lowest(self, n):
        got, free = [], (i for i, r in enumerate(self.refs) if r == 0)
        for i in free:
            if len(got) == n:
                break
            got.append(i)
        return got if len(got) == n else None

    def count(self, n):
        return -(-n // self.page)

    def cut(self, slot, new):
        for m in range(self.count(new), self.count(self.lens[slot])):
            self.refs[self.table[slot][m]] -= 1
            self.table[slot][m] = -1
        self.lens[slot] = new

    def grow(self, slots, want):
        told, full = [], False
        for slot, new in zip(slots, want):
            have = self.count(self.lens[slot])
            need = self.count(new) - have
            got = None if full and need else self.lowest(need)
            full = full or got is None
            told.append(0 if got is None else 1)
            if got is not None:
                for m, p in enumerate(got):
                    self.table[slot][have + m] = p
                    self.refs[p] = 1
                self.lens[slot] = new
        return told

    def tensors(self):
        return _ints(self.table), _ints(self.lens), _ints(self.refs)


def exact(case, seed):
    global own
    asked, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = asked
    op = case["op"]
    if op == "rope":
        out = []
        for x in (s["q"], s["k"]):
            y = _turned(x.reshape(-1, *x.shape[-2:]), s["positions"], case["rot"], case["inter"], case["scaling"],
                        case["dir"] == "bwd")
            out.append(y.view(x.shape))
        return out
    if op == "copy":
        out = []
        for c in (s["kc"], s["vc"]):
            c = c.double()
            for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
                c[:, b] = c[:, a]
            out.append(c)
        return out
    page = case["page"]
    book = _Book(s, page)
    if op in ("append", "tree"):
        cu = s["cu"].tolist()
        e = case["cache"] == "e4m3"
    if op == "append":
        q = _turned(s["q"], s["positions"], case["rot"], case["inter"])
        k = _turned(s["k"], s["positions"], case["rot"], case["inter"]) / (K_SCALE if e else 1)
        v = s["v"].double() / (V_SCALE if e else 1)
        kc, vc = s["kc"].double(), s["vc"].double()
        for b in range(case["B"]):
            n = cu[b + 1] - cu[b]
            at = [book.lens[b] - n + i for i in range(n)]
            pg = torch.tensor([book.table[b][p // page] for p in at], device=DEV)
            off = torch.tensor([p % page for p in at], device=DEV)
            kc[0, pg, off], vc[0, pg, off] = k[cu[b]:cu[b + 1]], v[cu[b]:cu[b + 1]]
        return q, kc, vc
    if op == "tree":
        T, Hq, d = s["q"].shape
        G = Hq // case["Hkv"]
        out, lses = torch.empty((T, Hq, d), dtype=torch.float64, device=DEV), torch.empty((Hq, T), dtype=torch.float64, device=DEV)
        for b in range(case["B"]):
            a, z, L = cu[b], cu[b + 1], book.lens[b]
            n = z - a
            pg = torch.tensor(book.table[b][:book.count(L)], device=DEV)
            seen = torch.ones((n, L), dtype=torch.bool, device=DEV)
            seen[:, L - n:] = s["mask"][a:z, :n] if s["mask"] is not None else torch.ones((n, n), dtype=torch.bool, device=DEV).tril()
            for h in range(case["Hkv"]):
                k = s["kc"][0, pg, :, h].reshape(-1, d)[:L].double() * (K_SCALE if e else 1)
                v = s["vc"][0, pg, :, h].reshape(-1, d)[:L].double() * (V_SCALE if e else 1)
                qh = s["q"][a:z, h * G:(h + 1) * G].double()
                x = (qh.reshape(n * G, d) @ k.t() / d ** 0.5).view(n, G, L)
                x = torch.where(seen[:, None], x, float("-inf"))
                l = torch.logsumexp(x, -1)
                out[a:z, h * G:(h + 1) * G] = ((x - l[..., None]).exp().view(n * G, L) @ v).view(n, G, d)
                lses[h * G:(h + 1) * G, a:z] = l.t()
        return out, lses
    slots = s["slots"].tolist()
    if op == "pages":
        for slot in slots:
            book.cut(slot, 0)
        told = book.grow(slots, s["want"].tolist())
        return (_ints(told), *book.tensors())
    kc, vc = s["kc"].double(), s["vc"].double()
    if op == "fork":
        dst = s["dst"].tolist()
        told = []
        for slot in dst:
            book.cut(slot, 0)
        full = False
        for a, b in zip(slots, dst):
            L = book.lens[a]
            got = None if full and L % page else book.lowest(1 if L % page else 0)
            full = full or got is None
            told.append(0 if got is None else 1)
            if got is None:
                continue
            for m in range(L // page):
                book.table[b][m] = book.table[a][m]
                book.refs[book.table[a][m]] += 1
            for p in got:
                book.table[b][L // page] = p
                book.refs[p] = 1
                for c in (kc, vc):
                    c[:, p, :L % page] = c[:, book.table[a][L // page], :L % page]
            book.lens[b] = L
        return (_ints(told), *book.tensors(), kc, vc)
    book.grow(slots, s["want"].tolist())
    cu, path, took = s["cu"].tolist(), s["path"].tolist(), s["took"].tolist()
    for b, slot in enumerate(slots):
        base = book.lens[slot] - (cu[b + 1] - cu[b])
        for i in range(took[b]):
            x, y = base + path[b][i], base + i
            for c in (kc, vc):
                c[:, book.table[slot][y // page], y % page] = c[:, book.table[slot][x // page], x % page]
        book.cut(slot, base + took[b])
    return (*book.tensors(), kc, vc)
