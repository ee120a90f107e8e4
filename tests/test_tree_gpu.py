"""Appending to the paged cache and attending over it, on the GPU, against the definition in 64
bits.

Tolerance of O.  The probabilities enter the second product rounded to bf16: 2^-8 relative
each, so 2^-8 A with A = sum p |v|.  O is rounded to bf16: 2^-8 |O|.  Scores are fp32 sums of d
<= 128 exact products: off by at most 2^-24 d sum |q k| scale <= 128 * 2^-24 * 128 * 0.64 * 0.09 =
6e-5 for unit normals, which moves a weight by twice that relative (numerator and sum): 1.2e-4
A; exponentials and fp32 sums stay below 5e-5 A.  So 2^-8 (A + |O|) + 2e-4 A.
An E4M3 cache: probabilities are two E4M3 terms.  The first leaves at most 2^-4 of p, the second
2^-4 of that: 2^-8 p; where p is so small that the terms are subnormal, each is off by at most half
the smallest step, 2^-10, together 2^-9.  Weights are stored times 2^4 relative to the row's
reference, a maximum taken earlier and never above the final one, so a row's sum is at least 2^4 sum
exp(s - max): an absolute 2^-9 / 2^4 F = 2^-13 F with F = sum |v| / sum exp(s - max).
LSE: the score error above, 6e-5, plus log and fp32 rounding at |LSE| < 20 (2e-6): 1e-4; queries
of an E4M3 cache are exact to 2^-17 of the row's largest: a score is off by a further 2^-17 * 4 *
sqrt(128) * 3 * 0.09 < 1e-4, and O by twice that of A."""
import math
import random

import pytest
import torch

import exact_attention_103_b200 as ea
import serve_ref as ref

pytestmark = pytest.mark.gpu
SCALES = {torch.bfloat16: (1.0, 1.0), torch.float8_e4m3fn: (0.0625, 0.03125)}


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def build(ctx, drafted, heads=2, d=128, page=16, dtype=torch.bfloat16, seed=0, layers=1, spare=3, fill=None):
    """A cache whose slot b holds ctx[b] + drafted[b] tokens on shuffled pages; what lies behind
    a sequence's end is `fill` (NaN where the type has it)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens = [c + n for c, n in zip(ctx, drafted)]
    counts = [-(-n // page) for n in lens]
    pages, width = sum(counts) + spare, max(max(counts), 1)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    table, refs, at = [], [0] * pages, 0
    for n in counts:
        table.append(order[at:at + n] + [-1] * (width - n))
        for p in order[at:at + n]:
            refs[p] = 1
        at += n
    ks, vs = SCALES[dtype]
    kv = []
    for s in (ks, vs):
        x = torch.full((layers, pages, page, heads, d), float("nan") if fill is None else fill, device="cuda").to(dtype)
        for row, n in zip(table, lens):
            for m in range(-(-n // page)):
                k = min(page, n - m * page)
                x[:, row[m], :k] = (torch.randn((layers, k, heads, d), generator=g, device="cuda") / s).to(dtype)
        kv.append(x)
    return ea.KVCache(kv[0], kv[1], ints(table), ints(lens), ints(refs), k_scale=ks, v_scale=vs)


def cu_of(drafted):
    return ints([0] + drafted).cumsum(0).to(torch.int32)


def tree_mask(drafted, seed, width=None, empty=0.0):
    r = random.Random(seed)
    width = width or max(drafted + [1])
    rows = []
    for n in drafted:
        m = torch.zeros(n, width, dtype=torch.bool)
        for i in range(n):
            p = r.randint(-1, i - 1)
            if p >= 0:
                m[i] = m[p]
            m[i, i] = True
        for i in range(n):
            if r.random() < empty:
                m[i] = False
        rows.append(m)
    return torch.cat(rows).cuda()


def verify(c, q, cu, mask, o, lse, slots=None, layer=0, scale=None):
    d = c.d
    scale = 1 / math.sqrt(d) if scale is None else scale
    f8 = c.dtype == torch.float8_e4m3fn
    cu, lens, table = cu.tolist(), c.lens.tolist(), c.page_table.tolist()
    for b in range(len(cu) - 1):
        a, z = cu[b], cu[b + 1]
        if a == z:
            continue
        s = b if slots is None else slots[b]
        L, n = lens[s], z - a
        k = ref.gather(c.k[layer], table[s], L, c.page_size).double() * c.k_scale
        v = ref.gather(c.v[layer], table[s], L, c.page_size).double() * c.v_scale
        seen = torch.ones(n, L, dtype=torch.bool, device="cuda")
        seen[:, L - n:] = torch.ones(n, n, dtype=torch.bool, device="cuda").tril() if mask is None else mask[a:z, :n].bool()
        wo, wl, A, F = ref.attend(q[a:z], k, v, seen, scale)
        got = o[a:z].double()
        assert torch.isfinite(got).all(), b
        tol = 2 ** -8 * (A + wo.abs()) + 2e-4 * A + (2 ** -13 * F + 2e-4 * A if f8 else 0) + 1e-30
        err = (got - wo).abs()
        assert (err <= tol).all(), (b, (err - tol).max().item(), (err / tol).max().item())
        gl, wl = lse[:, a:z].double().t(), wl
        none = torch.isinf(wl)
        assert torch.equal(gl[none], wl[none])
        assert ((gl - wl)[~none].abs() <= 1e-4 + (2 ** -17 * 4 * math.sqrt(128) * 3 * 0.09 if f8 else 0)).all(), (gl - wl)[~none].abs().max()


def run(c, drafted, Hq, mask=None, seed=1, **kw):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn((sum(drafted), Hq, c.d), generator=g, device="cuda").to(torch.bfloat16)
    cu = cu_of(drafted)
    o, lse = ea.tree_fwd(c, q, cu, mask=mask, **kw)
    ea.get_device_status()
    return q, cu, o, lse


KINDS = [(torch.bfloat16, 128), (torch.bfloat16, 64), (torch.float8_e4m3fn, 128), (torch.float8_e4m3fn, 64)]


@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("heads,G,page", [(1, 1, 16), (2, 4, 32), (3, 7, 128), (2, 16, 1024)])
def test_single_tokens(dtype, d, heads, G, page):
    """Decoding: contexts from nothing over tile edges to a few thousand."""
    ctx = [0, 1, 15, 126, 127, 128, 255, 256, 383, 1000, 2570]
    drafted = [1] * len(ctx)
    c = build(ctx, drafted, heads, d, page, dtype, seed=d + page)
    q, cu, o, lse = run(c, drafted, heads * G)
    verify(c, q, cu, None, o, lse)


@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("heads,G,page", [(2, 1, 64), (1, 4, 16), (2, 3, 32), (1, 8, 256)])
def test_trees(dtype, d, heads, G, page):
    """Ragged trees of 0 to 256 tokens, over one row tile and several, with rows that see nothing
    of their tree."""
    ctx = [0, 5, 64, 100, 127, 300, 1111, 40]
    drafted = [3, 1, 64, 0, 33, 128, 61, 256]
    c = build(ctx, drafted, heads, d, page, dtype, seed=d + page)
    mask = tree_mask(drafted, seed=page, empty=0.2)
    q, cu, o, lse = run(c, drafted, heads * G, mask)
    verify(c, q, cu, mask, o, lse)
    assert torch.isinf(lse[:, :3]).any() or mask[:3].any(1).all()


@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("G", [1, 4, 5, 128])
def test_chains(dtype, d, G):
    """Chunks of a prompt: causal among themselves, longer than any tile of rows."""
    ctx, drafted = [0, 77, 500, 0, 129], [1, 300, 129, 513, 2]
    if G == 128:
        ctx, drafted = [0, 77, 500], [1, 5, 3]
    c = build(ctx, drafted, 2, d, 16, dtype, seed=d + G)
    q, cu, o, lse = run(c, drafted, 2 * G)
    verify(c, q, cu, None, o, lse)


@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("G,n", [(1, 33), (1, 64), (3, 21), (5, 8), (8, 8), (16, 3), (33, 1), (64, 1)])
@pytest.mark.parametrize("masked", [False, True])
def test_rows_of_half_a_tile(dtype, d, G, n, masked):
    """33 to 64 rows, contexts that end before and behind the middle of a key tile."""
    ctx = [0, 1, 20, 63, 64, 65, 100, 128, 190, 700, 2100]
    drafted = [n] * len(ctx)
    c = build(ctx, drafted, 2, d, 64, dtype, seed=d + G)
    mask = tree_mask(drafted, seed=n, empty=0.2) if masked else None
    q, cu, o, lse = run(c, drafted, 2 * G, mask)
    verify(c, q, cu, mask, o, lse)


def test_rows_that_see_nothing():
    drafted = [4, 2]
    c = build([0, 0], drafted, 1)
    mask = torch.zeros(6, 4, dtype=torch.uint8, device="cuda")
    mask[2, 1] = 255
    q, cu, o, lse = run(c, drafted, 3, mask)
    verify(c, q, cu, mask, o, lse)
    assert (o[[0, 1, 3, 4, 5]] == 0).all() and torch.isinf(lse[:, [0, 1, 3, 4, 5]]).all() and torch.isfinite(lse[:, 2]).all()


@pytest.mark.parametrize("dtype", list(SCALES))
def test_long_context_and_peaked_scores(dtype):
    """Keys that grow along the sequence move the running maximum again and again; some rows'
    weights sit on one key."""
    ctx, drafted = [20011, 4097], [17, 2]
    c = build(ctx, drafted, 2, 128, 64, dtype, seed=9)
    for b in range(2):
        L = ctx[b] + drafted[b]
        row = c.page_table[b].tolist()
        for m in range(-(-L // 64)):
            x = c.k[0, row[m]].float() * (0.05 + 2.0 * m * 64 / L)
            c.k[0, row[m]] = x.to(dtype)
    mask = tree_mask(drafted, 3)
    q, cu, o, lse = run(c, drafted, 8, mask)
    d = 128
    f8 = dtype == torch.float8_e4m3fn
    table, lens = c.page_table.tolist(), c.lens.tolist()
    cul = cu.tolist()
    for b in range(2):  # the score error grows with the keys: twice the unit normals' bound
        a, z, L = cul[b], cul[b + 1], lens[b]
        k = ref.gather(c.k[0], table[b], L, 64).double() * c.k_scale
        v = ref.gather(c.v[0], table[b], L, 64).double() * c.v_scale
        seen = torch.ones(z - a, L, dtype=torch.bool, device="cuda")
        seen[:, L - (z - a):] = mask[a:z, :z - a]
        wo, wl, A, F = ref.attend(q[a:z], k, v, seen, 1 / math.sqrt(d))
        tol = 2 ** -8 * (A + wo.abs()) + 4e-4 * A + (2 ** -13 * F + 2e-3 * A if f8 else 0)
        assert ((o[a:z].double() - wo).abs() <= tol).all()
        assert (lse[:, a:z].double().t() - wl).abs().max() <= 2e-4 + (8e-4 if f8 else 0)


def test_slots_layers_and_shared_sequences():
    """Sequences in any order of slots, one slot twice, a layer in the middle."""
    ctx, held = [50, 200, 7, 129], [9, 9, 9, 9]
    c = build(ctx, held, 2, 64, 32, layers=3, seed=5)
    slots, drafted = [3, 1, 3], [9, 4, 9]
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn((22, 4, 64), generator=g, device="cuda").to(torch.bfloat16)
    cu = cu_of(drafted)
    for layer in range(3):
        o, lse = ea.tree_fwd(c, q, cu, slots=ints(slots), layer=layer, scale=0.3)
        verify(c, q, cu, None, o, lse, slots, layer, 0.3)
    ea.get_device_status()


def test_many_sequences():
    r = random.Random(1)
    ctx = [r.choice([0, r.randint(0, 40), r.randint(0, 700)]) for _ in range(1024)]
    drafted = [r.choice([0, 1, 1, 2, 5]) for _ in ctx]
    ctx = [c if n else 0 for c, n in zip(ctx, drafted)]
    c = build(ctx, drafted, 1, 64, 16, seed=6)
    q, cu, o, lse = run(c, drafted, 2)
    verify(c, q, cu, None, o, lse)


@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("masked", [False, True])
def test_many_tiles_and_mixed_rows(dtype, d, masked):
    """Every SM takes dozens of key tiles of many items, whose rows fill from a part of a tile to
    several, one kind behind another."""
    r = random.Random(d)
    ctx = [r.randint(0, 3000) for _ in range(40)]
    drafted = [r.choice([1, 1, 3, 16, 17, 33, 64, 130]) for _ in ctx]
    c = build(ctx, drafted, 8, d, 32, dtype, seed=11)
    mask = tree_mask(drafted, 5) if masked else None
    q, cu, o, lse = run(c, drafted, 32, mask)
    verify(c, q, cu, mask, o, lse)
    for _ in range(3):
        o2, l2 = ea.tree_fwd(c, q, cu, mask=mask)
        assert torch.equal(o, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("dtype,d", KINDS)
def test_long_batches_of_single_tokens(dtype, d):
    r = random.Random(d)
    ctx = [r.randint(500, 6000) for _ in range(48)]
    drafted = [1] * 48
    c = build(ctx, drafted, 8, d, 64, dtype, seed=12)
    q, cu, o, lse = run(c, drafted, 16)
    verify(c, q, cu, None, o, lse)


@pytest.mark.parametrize("dtype", list(SCALES))
def test_1024_sequences(dtype):
    """As many sequences as a batch holds, some of them without a token."""
    r = random.Random(3)
    drafted = [r.choice([0, 1, 1, 2, 7]) for _ in range(1024)]
    ctx = [r.randint(0, 90) for _ in drafted]
    c = build(ctx, drafted, 1, 64, 16, dtype, seed=13)
    q, cu, o, lse = run(c, drafted, 4)
    verify(c, q, cu, None, o, lse)


@pytest.mark.parametrize("cu", [[0, 3, 2, 6], [0, 3, 6, 7], [-1, 2, 4, 6]])
def test_offsets_that_decrease_or_leave_the_batch(cu):
    c = build([20, 5, 9], [3, 3, 3], 1, 64, 16)
    q = torch.randn(6, 2, 64, device="cuda").to(torch.bfloat16)
    o, lse = torch.full_like(q, 7.0), torch.full((2, 6), 7.0, device="cuda")
    ea.tree_fwd(c, q, ints(cu), out=o, lse=lse)
    assert (o == 7).all() and (lse == 7).all()
    with pytest.raises(ea.AttnError):
        ea.get_device_status()


def test_rows_outside_the_batch_stay():
    c = build([100, 30], [3, 2], 1, 128, 16)
    q = torch.randn(12, 2, 128, device="cuda").to(torch.bfloat16)
    cu = ints([2, 5, 7])  # rows 0, 1 and 7.. belong to no sequence
    o, lse = torch.full_like(q, 7.0), torch.full((2, 12), 7.0, device="cuda")
    ea.tree_fwd(c, q, cu, out=o, lse=lse)
    ea.get_device_status()
    for rows in (slice(0, 2), slice(7, 12)):
        assert (o[rows] == 7).all() and (lse[:, rows] == 7).all()
    sub = ea.tree_fwd(c, q[2:7].contiguous(), ints([0, 3, 5]))
    assert torch.equal(o[2:7], sub[0]) and torch.equal(lse[:, 2:7], sub[1])


def test_bad_pages_and_lengths_are_reported():
    """A sequence the tables do not describe leaves its rows alone, the others are computed."""
    c = build([100, 30, 60], [3, 3, 3], 1, 128, 16)
    q = torch.randn(9, 2, 128, device="cuda").to(torch.bfloat16)
    cu = ints([0, 3, 6, 9])
    want = ea.tree_fwd(c, q, cu)
    ea.get_device_status()

    def again(**kw):
        o, lse = torch.full_like(q, 7.0), torch.full((2, 9), 7.0, device="cuda")
        ea.tree_fwd(c, q, cu, out=o, lse=lse, **kw)
        with pytest.raises(ea.AttnError) as e:
            ea.get_device_status()
        assert e.value.status == ea.ATTN_ERR_INVALID_ARG
        assert torch.equal(o[:3], want[0][:3]) and torch.equal(o[6:], want[0][6:])
        return o, lse
    c.lens[1] = 2  # fewer than its drafted tokens
    assert (again()[0][3:6] == 7).all()
    c.lens[1] = 10 ** 6
    assert (again()[0][3:6] == 7).all()
    c.lens[1] = 33
    assert (again(slots=ints([0, -1, 2]))[0][3:6] == 7).all()
    assert (again(slots=ints([0, 3, 2]))[0][3:6] == 7).all()
    keep = c.page_table.clone()
    for page in (-1, c.pages, 2 ** 30):
        c.page_table[1, 1] = page
        again()
        c.page_table.copy_(keep)
    mask = torch.ones(9, 2, dtype=torch.bool, device="cuda")  # narrower than the drafts
    o, lse = torch.full_like(q, 7.0), torch.full((2, 9), 7.0, device="cuda")
    ea.tree_fwd(c, q, cu, mask=mask, out=o, lse=lse)
    assert (o == 7).all()
    with pytest.raises(ea.AttnError):
        ea.get_device_status()


def test_repeatable_on_streams_and_in_graphs():
    ctx, drafted = [3000, 50, 777], [20, 20, 20]
    c = build(ctx, drafted, 2, 128, 32)
    mask = tree_mask(drafted, 4)
    q, cu, o, lse = run(c, drafted, 8, mask)
    for _ in range(3):
        o2, l2 = ea.tree_fwd(c, q, cu, mask=mask)
        assert torch.equal(o, o2) and torch.equal(lse, l2)
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for i, s in enumerate(streams * 4):  # calls at the same time, each with its own workspace
        s.wait_stream(torch.cuda.current_stream())
        got.append(ea.tree_fwd(c, q, cu, mask=mask, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(o, x) and torch.equal(lse, y) for x, y in got)
    graphs, held = [], []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            held.append(ea.tree_fwd(c, q, cu, mask=mask))
    q.mul_(0.5)
    want = ea.tree_fwd(c, q, cu, mask=mask)
    torch.cuda.synchronize()
    for i, s in zip((0, 1, 0, 1), streams + streams[:1]):
        with torch.cuda.stream(s):
            graphs[i].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(want[0], x) and torch.equal(want[1], y) for x, y in held)
    ea.get_device_status()


@pytest.mark.parametrize("dtype", list(SCALES))
def test_one_slot_for_two_sequences_layers_and_scales(dtype):
    """Reading is shared freely: two sequences of a call may be the same slot, in any layer, with any
    scale; a strided cache of several layers is read in place."""
    c = build([300, 40], [5, 5], 2, 128, 32, dtype, seed=21, layers=3)
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn((15, 8, 128), generator=g, device="cuda").to(torch.bfloat16)
    q[5:10] = q[:5]
    cu = ints([0, 5, 10, 15])
    # scales below 1 / sqrt(d), which the tolerances assume; the two sequences need not be bitwise
    # alike, as their keys may be split over the SMs at different places
    for layer, scale in ((2, 0.05), (0, 0.02)):
        o, lse = ea.tree_fwd(c, q, cu, slots=ints([0, 0, 1]), layer=layer, scale=scale)
        ea.get_device_status()
        verify(c, q, cu, None, o, lse, slots=[0, 0, 1], layer=layer, scale=scale)


def test_append_in_place_and_page_calls_on_another_stream():
    heads, d, page = 2, 128, 16
    plan = ea.Rope(d)
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn((9, h, d), generator=g, device="cuda").to(torch.bfloat16) for h in (8, heads, heads))
    cu, slots, want = ints([0, 4, 9]), ints([1, 2]), ints([20, 33])
    caches, outs = [], []
    side = torch.cuda.Stream()
    for stream in (None, side):
        c = ea.KVCache.empty(1, 20, page, heads, d, 4, 8)
        c.k.zero_(), c.v.zero_()
        torch.cuda.synchronize()
        x = q.clone()
        side.wait_stream(torch.cuda.current_stream())
        assert c.alloc(slots, want, stream=stream) is not None
        y = ea.rope_append(c, x, k, v, cu, plan=plan, slots=slots, out=x, stream=stream)
        assert y is x
        c.fork(ints([1]), ints([3]), stream=stream)
        o, lse = ea.tree_fwd(c, x, cu, slots=slots, stream=stream)
        c.compact(cu, ints([[0, 3], [4, -1]]), ints([2, 1]), slots=slots, stream=stream)
        c.free(ints([3]), stream=stream)
        torch.cuda.synchronize()
        ea.get_device_status()
        caches.append(c)
        outs.append((x, o, lse))
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    for name in ("k", "v", "page_table", "lens", "refs"):
        assert torch.equal(getattr(caches[0], name), getattr(caches[1], name))
    turned = ea.rope_fwd(plan, q, positions=torch.cat([torch.arange(16, 20), torch.arange(28, 33)]).to(torch.int32).cuda(),
                         cu_seqlens=cu)
    assert torch.equal(outs[0][0], turned)


def test_a_step_in_a_graph():
    """Pages, append, attention and compaction of a decoding step, captured once and replayed on
    another stream: every replay continues from the state that the last one left."""
    heads, G, d, page, n = 2, 4, 64, 16, 6
    plan = ea.Rope(d)
    g = torch.Generator(device="cuda").manual_seed(5)
    start = [37, 16, 90]
    T = n * len(start)
    q, k, v = (torch.randn((T, h, d), generator=g, device="cuda").to(torch.bfloat16) for h in (heads * G, heads, heads))
    cu, slots = ints([n * i for i in range(len(start) + 1)]), ints([2, 0, 1])
    mask = tree_mask([n] * len(start), 6)
    path, took = ints([[0, 2, 5], [1, -1, -1], [-1, -1, -1]]), ints([3, 1, 0])
    other = ints([4])

    def fresh():
        g = torch.Generator(device="cuda").manual_seed(7)
        c = ea.KVCache.empty(1, 60, page, heads, d, 5, 12)
        for x in (c.k, c.v):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda").to(torch.bfloat16))
        c.alloc(ints([0, 1, 2]), ints(start))
        c.fork(ints([0]), other)
        return c, ints([0] * 3)

    def step(c, want):
        want.copy_(c.lens[slots.long()] + n)
        granted = c.alloc(slots, want)
        turned = ea.rope_append(c, q, k, v, cu, plan=plan, slots=slots)
        o, lse = ea.tree_fwd(c, turned, cu, mask=mask, slots=slots)
        c.compact(cu, path, took, slots=slots)
        c.free(other)
        fork = c.fork(ints_at(slots, 1), other)
        return granted, turned, o, lse, fork

    def ints_at(t, i):
        return t[i:i + 1]

    eager, want = fresh()
    seen = []
    for _ in range(4):
        seen.append([x.clone() for x in step(eager, want)] + [x.clone() for x in (eager.lens, eager.refs)])
    c, want = fresh()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    keep = [x.clone() for x in (c.page_table, c.lens, c.refs, c.k, c.v)]
    step(c, want)  # once outside, then back
    for x, y in zip((c.page_table, c.lens, c.refs, c.k, c.v), keep):
        x.copy_(y)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = step(c, want)
    s = torch.cuda.Stream()
    for i in range(4):
        with torch.cuda.stream(s):
            graph.replay()
        s.synchronize()
        for x, y in zip(list(out) + [c.lens, c.refs], seen[i]):
            assert torch.equal(x, y)
    assert torch.equal(c.k, eager.k) and torch.equal(c.v, eager.v)
    ea.get_device_status()


@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("dim,inter,page", [(None, False, 16), (64, True, 64), (32, False, 32)])
def test_append(dtype, d, dim, inter, page):
    """New tokens land in their rows, rotated and rounded once; every other byte stays."""
    ctx, drafted, heads, Hq = [0, 15, 130, 9, 64], [1, 2, 40, 0, 77], 3, 6
    c = build(ctx, drafted, heads, d, page, dtype, layers=2, seed=8, fill=1.0)
    T = sum(drafted)
    g = torch.Generator(device="cuda").manual_seed(3)
    qkv = torch.randn((T, Hq + 2 * heads, d), generator=g, device="cuda").to(torch.bfloat16)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + heads], qkv[:, Hq + heads:]
    plan = None if dim is None else ea.Rope(dim, interleaved=inter)
    cu, perm = cu_of(drafted), [4, 2, 0, 3, 1]  # sequence i of this call is slot perm[i]
    order = [drafted[s] for s in perm]
    cu = cu_of(order)
    before = c.k.clone(), c.v.clone()
    pos = torch.cat([torch.arange(ctx[s], ctx[s] + drafted[s]) for s in perm]).cuda()
    for given in (None, (pos * 3 + 1).to(torch.int32)):
        got = ea.rope_append(c, q, k, v, cu, plan=plan, positions=given, slots=ints(perm), layer=1)
        ea.get_device_status()
        at = pos if given is None else given
        if plan is None:
            wq, wk = q.double(), k.double()
        else:
            f, amp = ref.rope_freqs(dim)
            wq, wk = (ref.rope(x.double(), at, f.cuda(), amp, inter) for x in (q, k))
        # see test_rope_gpu for 4e-7 of the pair (below 12 for these); E4M3's eps/2 is 2^-4, its
        # smallest half step 2^-10
        assert ((got.double() - wq).abs() <= 2 ** -8 * wq.abs() + 5e-6).all()
        kc, vc = before[0].clone(), before[1].clone()
        rows = []
        for i, s in enumerate(perm):
            rows += [int(c.page_table[s, p // page]) * page + p % page for p in range(ctx[s], ctx[s] + drafted[s])]
        rows = torch.tensor(rows, device="cuda")
        flat_k, flat_v = c.k[1].flatten(0, 1), c.v[1].flatten(0, 1)
        if dtype == torch.bfloat16:
            assert ((flat_k[rows].double() - wk).abs() <= 2 ** -8 * wk.abs() + 5e-6).all()
            assert torch.equal(flat_v[rows], v)
        else:
            for flat, w, s in ((flat_k, wk, c.k_scale), (flat_v, v.double(), c.v_scale)):
                w = (w / s).clamp(-448, 448)
                assert ((flat[rows].double() - w).abs() <= 2 ** -4 * w.abs() + 2 ** -10 + 5e-6 / s).all()
        for t, b in ((c.k, before[0]), (c.v, before[1])):
            x, y = t.view(torch.uint8).clone(), b.view(torch.uint8).clone()
            x[1].flatten(0, 1)[rows], y[1].flatten(0, 1)[rows] = 0, 0
            assert torch.equal(x, y)


def test_append_refuses_on_the_device():
    c = build([4, 4], [3, 3], 1, 64, 16, fill=2.0)
    x = torch.randn(6, 1, 64, device="cuda").to(torch.bfloat16)
    for kw in (dict(slots=ints([0, 0])), dict(slots=ints([0, 9]))):
        k0 = c.k.clone()
        ea.rope_append(c, None, x, x, ints([0, 3, 6]), **kw)
        with pytest.raises(ea.AttnError):
            ea.get_device_status()
        first = int(c.page_table[0, 0])
        assert torch.equal(c.k[0, first, 4:7], x[:3])
        k0[0, first, 4:7] = x[:3]
        assert torch.equal(c.k, k0)
        c.k[0, first, 4:7] = 0
    c.lens[1] = 2
    k0 = c.k.clone()
    ea.rope_append(c, None, x, x, ints([0, 3, 6]))
    with pytest.raises(ea.AttnError):
        ea.get_device_status()
    k0[0, int(c.page_table[0, 0]), 4:7] = x[:3]
    assert torch.equal(c.k, k0)


@pytest.mark.parametrize("dtype", list(SCALES))
def test_a_serving_run(dtype):
    """Prompt in two chunks, three drafted trees verified and compacted, a fork, single tokens:
    each step against plain attention over the tokens that should be there."""
    ks, vs = SCALES[dtype]
    heads, G, d, page, layers = 2, 4, 64, 16, 2
    c = ea.KVCache.empty(layers, 60, page, heads, d, 4, 20, dtype=dtype, k_scale=ks, v_scale=vs)
    plan = ea.Rope(d)
    f, amp = ref.rope_freqs(d)
    g = torch.Generator(device="cuda").manual_seed(1)
    r = random.Random(1)
    K = [[torch.zeros(0, heads, d, device="cuda").to(dtype) for _ in range(layers)] for _ in range(4)]
    V = [[torch.zeros(0, heads, d, device="cuda").to(dtype) for _ in range(layers)] for _ in range(4)]

    def step(slots, new, mask=None, depth=None):
        have = [K[s][0].shape[0] for s in slots]
        assert c.alloc(ints(slots), ints([h + n for h, n in zip(have, new)])).tolist() == [1] * len(slots)
        cu, T = cu_of(new), sum(new)
        pos = None
        at = torch.cat([torch.arange(h, h + n) for h, n in zip(have, new)]).cuda()
        if depth is not None:
            at = torch.cat([torch.tensor(x) + h for x, h in zip(depth, have)]).cuda()
            pos = at.to(torch.int32)
        for l in range(layers):
            qkv = torch.randn((T, heads * (G + 2), d), generator=g, device="cuda").to(torch.bfloat16)
            q, k, v = qkv[:, :heads * G], qkv[:, heads * G:heads * (G + 1)], qkv[:, heads * (G + 1):]
            q2 = ea.rope_append(c, q, k, v, cu, plan=plan, positions=pos, slots=ints(slots), layer=l)
            o, lse = ea.tree_fwd(c, q2, cu, mask=mask, slots=ints(slots), layer=l)
            wk = ref.rope(k.double(), at, f.cuda(), amp, False)
            a = 0
            for s, n in zip(slots, new):
                table = c.page_table[s].tolist()
                kk = ref.gather(c.k[l], table, K[s][l].shape[0] + n, page)
                vv = ref.gather(c.v[l], table, K[s][l].shape[0] + n, page)
                assert torch.equal(kk[:-n].view(torch.uint8), K[s][l].view(torch.uint8))  # what was there still is
                near = (kk[-n:].double() * ks - wk[a:a + n]).abs()
                eps = 2 ** -8 if dtype == torch.bfloat16 else 2 ** -4
                assert (near <= eps * wk[a:a + n].abs() + 2 ** -10 * ks + 5e-6).all()
                K[s][l], V[s][l] = kk, vv
                a += n
            verify(c, q2, cu, mask, o, lse, slots, l)

    step([2, 0], [50, 33])
    step([2, 0, 1], [30, 1, 20])
    for _ in range(3):
        new = [r.randint(2, 30) for _ in range(3)]
        mask = tree_mask(new, r.random())
        step([0, 2, 1], new, mask, [(mask[sum(new[:i]):sum(new[:i + 1])].sum(1) - 1).tolist() for i in range(3)])
        path = [sorted(r.sample(range(n), r.randint(0, n))) for n in new]
        width = max(1, max(map(len, path)))
        c.compact(cu_of(new), ints([p + [-1] * (width - len(p)) for p in path]), ints([len(p) for p in path]), slots=ints([0, 2, 1]))
        for s, n, p in zip([0, 2, 1], new, path):
            for l in range(layers):
                for X in (K, V):
                    keep = X[s][l].shape[0] - n
                    X[s][l] = torch.cat([X[s][l][:keep].view(torch.uint8), X[s][l][keep:].view(torch.uint8)[p]]).view(dtype)
    assert c.fork(ints([2]), ints([3])).tolist() == [1]
    for X in (K, V):
        X[3] = [x.clone() for x in X[2]]
    for _ in range(3):
        step([3, 2, 0, 1], [1, 1, 1, 1])
    c.free(ints([0, 1, 2, 3]))
    assert (c.refs == 0).all() and (c.page_table == -1).all()
    ea.get_device_status()
