"""The serving operators' argument checks, without a GPU: the C ABI refuses before it touches
the device, and the Python binding before it calls the library."""
import ctypes
import math

import pytest
import torch

import exact_attention_103_b200 as ea
from exact_attention_103_b200 import build as ea_build
from exact_attention_103_b200 import cache as ec

FAKE = 0x10000  # aligned, never dereferenced: validation returns first
BAD, NO, WS = ea.ATTN_ERR_INVALID_ARG, ea.ATTN_ERR_UNSUPPORTED, ea.ATTN_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    ea_build.build()
    return ea.load_library()


def view(**kw):
    base = dict(k=FAKE, v=FAKE, page_table=FAKE, lens=FAKE, refs=FAKE, layers=2, pages=8, page_size=16,
                heads=4, d=128, slots=3, max_pages=5, e4m3=0, k_scale=1.0, v_scale=1.0)
    base.update(kw)
    return ec.CacheView(*(base[n] for n, _ in ec.CacheView._fields_))


def plan(**kw):
    base = dict(turns=FAKE, dim=64, interleaved=0, amplitude=1.0)
    base.update(kw)
    return ec.RopePlan(*(base[n] for n, _ in ec.RopePlan._fields_))


def rows(**kw):
    base = dict(src=FAKE, dst=FAKE, heads=4, src_batch=0, src_token=512, src_head=128, dst_batch=0,
                dst_token=512, dst_head=128)
    base.update(kw)
    return ec.Rows(*(base[n] for n, _ in ec.Rows._fields_))


@pytest.mark.parametrize("kw,want", [
    (dict(d=96), NO), (dict(page_size=8), NO), (dict(page_size=24), NO), (dict(page_size=2048), NO),
    (dict(slots=8193), NO), (dict(layers=0), BAD), (dict(pages=0), BAD), (dict(heads=-1), BAD),
    (dict(k=None), BAD), (dict(k=FAKE + 8), BAD), (dict(lens=None), BAD), (dict(refs=FAKE + 2), BAD),
    (dict(e4m3=2), BAD), (dict(e4m3=1, k_scale=0.0), BAD), (dict(v_scale=math.nan), BAD),
    (dict(pages=1 << 27, page_size=64), NO), (dict(max_pages=1 << 27, page_size=64), NO)])
def test_cache_checks_reach_every_operator(lib, kw, want):
    c = ctypes.byref(view(**kw))
    r = ctypes.byref(rows())
    assert lib.attn_cache_alloc(c, FAKE, FAKE, 1, FAKE, None) == want
    assert lib.attn_cache_free(c, FAKE, 1, None) == want
    assert lib.attn_cache_fork(c, FAKE, FAKE, 1, FAKE, FAKE, 16, None) == want
    assert lib.attn_cache_copy(c, FAKE, FAKE, 1, None) == want
    assert lib.attn_cache_compact(c, FAKE, FAKE, 1, FAKE, None, 1, None) == want
    assert lib.attn_rope_append(c, 0, None, r, r, r, 1, 1, FAKE, None, None, None) == want
    assert lib.attn_tree_fwd(c, 0, FAKE, FAKE, FAKE, 4, 1, 1, FAKE, None, None, 0, 0.1, FAKE, 1 << 30, None) == want


def test_page_operations_refuse(lib):
    c = ctypes.byref(view())
    assert lib.attn_cache_alloc(None, FAKE, FAKE, 1, FAKE, None) == BAD
    assert lib.attn_cache_alloc(c, None, FAKE, 1, FAKE, None) == BAD
    assert lib.attn_cache_alloc(c, FAKE, FAKE + 1, 1, FAKE, None) == BAD
    assert lib.attn_cache_alloc(c, FAKE, FAKE, 8193, FAKE, None) == BAD
    assert lib.attn_cache_alloc(c, FAKE, FAKE, -1, FAKE, None) == BAD
    assert lib.attn_cache_free(c, None, 2, None) == BAD
    assert lib.attn_cache_fork(c, FAKE, FAKE, 2, FAKE, FAKE, 16, None) == WS
    assert lib.attn_cache_fork(c, FAKE, FAKE, 2, FAKE, None, 64, None) == WS
    assert lib.attn_cache_fork(c, FAKE, FAKE, 2, FAKE, FAKE + 8, 64, None) == WS
    assert lib.attn_cache_fork_workspace_size(3) == 48 and lib.attn_cache_fork_workspace_size(-1) == 0
    assert lib.attn_cache_copy(c, FAKE, None, 2, None) == BAD
    assert lib.attn_cache_compact(c, FAKE, None, 1, FAKE, None, 1, None) == BAD
    assert lib.attn_cache_compact(c, FAKE, FAKE, 1, FAKE, None, 4, None) == BAD  # more sequences than slots
    assert lib.attn_cache_compact(c, FAKE, FAKE, 1, FAKE, FAKE, 1025, None) == NO
    for st in (lib.attn_cache_alloc(c, None, None, 0, None, None), lib.attn_cache_free(c, None, 0, None),
               lib.attn_cache_fork(c, None, None, 0, None, None, 0, None), lib.attn_cache_copy(c, None, None, 0, None),
               lib.attn_cache_compact(c, None, None, 0, None, None, 0, None)):
        assert st == ea.ATTN_OK  # nothing to do


def test_rope_refuses(lib):
    def call(p=plan(), type=0, t=(rows(), rows()), count=2, d=128, B=1, N=4, cu=None, pos=None):
        two = (ec.Rows * 2)(*t)
        return lib.attn_rope(None if p is None else ctypes.byref(p), 0, type, two, count, d, B, N, cu, pos, None)
    assert call(p=None) == BAD and call(p=plan(turns=None)) == BAD and call(p=plan(turns=FAKE + 4)) == BAD
    assert call(p=plan(dim=24)) == NO and call(p=plan(dim=256)) == NO and call(p=plan(dim=0)) == NO
    assert call(p=plan(amplitude=0.0)) == BAD and call(p=plan(amplitude=math.inf)) == BAD
    assert call(type=3) == NO and call(d=72) == NO and call(d=272) == NO
    assert call(count=3) == BAD and call(count=0) == BAD and call(B=-1) == BAD and call(N=-1) == BAD
    assert call(t=(rows(src=None), rows())) == BAD and call(t=(rows(), rows(dst=FAKE + 8))) == BAD
    assert call(t=(rows(src_head=4), rows())) == BAD and call(t=(rows(dst_token=1), rows())) == BAD
    assert call(t=(rows(src_batch=9), rows())) == BAD and call(t=(rows(heads=0), rows())) == BAD
    assert call(type=2, t=(rows(src_head=132), rows(src_head=132)), pos=FAKE + 1) == BAD
    assert call(cu=FAKE + 2) == BAD and call(cu=FAKE, B=1025) == NO
    assert call(B=1 << 20, N=1 << 12) == NO
    assert call(B=0) == ea.ATTN_OK and call(N=0) == ea.ATTN_OK


def test_append_refuses(lib):
    def call(layer=0, p=None, q=rows(), k=rows(), v=rows(), B=1, T=4, cu=FAKE, slots=None, pos=None):
        r = [None if x is None else ctypes.byref(x) for x in (p, q, k, v)]
        return lib.attn_rope_append(ctypes.byref(view()), layer, *r, B, T, cu, slots, pos, None)
    assert call(layer=2) == BAD and call(layer=-1) == BAD and call(B=-1) == BAD and call(T=-1) == BAD
    assert call(B=1025, slots=FAKE) == NO and call(B=4) == BAD  # 3 slots
    assert call(k=None) == BAD and call(v=None) == BAD and call(k=rows(heads=3)) == BAD
    assert call(p=plan(dim=200)) == NO and call(cu=None) == BAD and call(pos=FAKE + 2) == BAD
    assert call(q=rows(dst=None)) == BAD and call(v=rows(src_token=500)) == BAD
    assert call(B=0) == ea.ATTN_OK and call(T=0) == ea.ATTN_OK


def test_tree_refuses(lib):
    need = lib.attn_tree_workspace_size(128)

    def call(layer=0, q=FAKE, lse=FAKE, Hq=8, B=1, T=4, cu=FAKE, slots=None, mask=None, width=0, scale=0.1,
             ws=FAKE, size=1 << 40):
        return lib.attn_tree_fwd(ctypes.byref(view()), layer, q, FAKE, lse, Hq, B, T, cu, slots, mask, width, scale,
                                 ws, size, None)
    assert call(layer=2) == BAD and call(Hq=6) == NO and call(Hq=0) == NO and call(Hq=4 * 129) == NO
    assert call(B=-1) == BAD and call(T=-1) == BAD and call(B=1025, slots=FAKE) == NO and call(B=4) == BAD
    assert call(scale=0.0) == BAD and call(scale=math.nan) == BAD
    assert call(mask=FAKE, width=0) == NO and call(mask=FAKE, width=257) == NO
    assert call(q=None) == BAD and call(q=FAKE + 8) == BAD and call(lse=FAKE + 2) == BAD
    assert call(cu=None) == BAD and call(slots=FAKE + 1) == BAD
    if need:
        assert call(size=need - 1) == WS and call(ws=None) == WS and call(ws=FAKE + 128) == WS
    assert call(T=1 << 30, Hq=8) == NO
    assert call(B=0) == ea.ATTN_OK and call(T=0) == ea.ATTN_OK


@pytest.mark.parametrize("kw", [dict(dim=0), dict(dim=24), dict(dim=64, base=1.0), dict(dim=64, factor=0.5),
                                dict(dim=64, scaling="cubic"), dict(dim=64, scaling="yarn", factor=2.0),
                                dict(dim=64, scaling="yarn", factor=2.0, original_len=64, beta_fast=1.0),
                                dict(dim=64, amplitude=0.0), dict(dim=64, amplitude=math.nan)])
def test_rope_plan_refuses(kw):
    with pytest.raises(ValueError):
        ea.Rope(device="cpu", **kw)


@pytest.mark.parametrize("kw", [dict(dim=128), dict(dim=64, scaling="linear", factor=4.0),
                                dict(dim=64, scaling="ntk", factor=4.0),
                                dict(dim=128, scaling="yarn", factor=8.0, original_len=4096)])
def test_rope_plan_fractions(kw):
    """The fixed-point fractions are the frequencies: relatively off by the doubles they come from
    (pow, two products and a division: below 2^-48), absolutely by half a unit of the fixed
    point, 2^-65 turns = 2^-65 * 2 pi radians (which for a frequency of 1.4e-5 is 2^-47 of it)."""
    import serve_ref
    p = ea.Rope(device="cpu", **kw)
    f, amp = serve_ref.rope_freqs(kw["dim"], 10000.0, kw.get("scaling"), kw.get("factor", 1.0), kw.get("original_len"))
    got = p.turns.double() / 2.0 ** 64 * 2 * math.pi
    assert torch.allclose(got, f, rtol=2 ** -48, atol=2 ** -65 * 2 * math.pi) and (p.turns > 0).all()
    assert p.amplitude == pytest.approx(amp, rel=1e-15)


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    p = ea.Rope(64, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        ea.rope_fwd(p, x)
    with pytest.raises(ValueError, match="CUDA"):
        ea.KVCache(x, x, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                   torch.zeros(1, dtype=torch.int32))
