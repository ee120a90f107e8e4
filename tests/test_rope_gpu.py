"""Rotary positions on the GPU against the definition in 64 bits: forward and gradient, both
pair layouts, part of a head, scaled contexts, types, strides, packed batches.

Tolerance: a result is a cos - b sin in fp32, rounded once to its type.  The angle is off
by at most 2^-25 turns of pi (the 32-bit fraction read as fp32: 1e-7), sine and cosine by 2
ulp (1.2e-7), and two products and a sum round three times (1.8e-7): 4e-7 (|a| + |b|)
amplitude in all; the rounding to the type adds eps/2 relative to the result, and below the
type's smallest normal number half its smallest step, which is smallest_normal * eps / 2 (fp16:
2^-14 * 2^-11 = 2^-25 = 3e-8, above the eps/2 of a result of 1e-5, 2^-11 * 1e-5 = 5e-9)."""
import pytest
import torch

import exact_attention_103_b200 as ea
import serve_ref as ref

pytestmark = pytest.mark.gpu


def check(got, want, x, dim, inter, amp):
    want = want.double()
    size = x.double().abs()
    pair = size.clone()
    if inter:
        s = size[..., 0:dim:2] + size[..., 1:dim:2]
        pair[..., 0:dim:2], pair[..., 1:dim:2] = s, s
    else:
        s = size[..., :dim // 2] + size[..., dim // 2:dim]
        pair[..., :dim // 2], pair[..., dim // 2:dim] = s, s
    fi = torch.finfo(got.dtype)
    tol = fi.eps / 2 * want.abs().clamp(min=fi.smallest_normal) + 4e-7 * pair * amp
    tol[..., dim:] = 0  # what passes through is not touched
    err = (got.double() - want).abs()
    assert got.shape == want.shape and torch.isfinite(got).all()
    assert (err <= tol).all(), (err - tol).max().item()


def rand(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,dim,Hq,Hk", [(128, 128, 5, 2), (64, 32, 7, 1), (128, 16, 1, 1), (80, 48, 3, 3), (256, 256, 2, 1)])
def test_dense(dtype, inter, d, dim, Hq, Hk):
    q, k = rand((3, 37, Hq, d), dtype, 1), rand((3, 37, Hk, d), dtype, 2)
    plan = ea.Rope(dim, interleaved=inter)
    f, amp = ref.rope_freqs(dim)
    pos = torch.arange(37, device="cuda").expand(3, 37)
    f = f.cuda()
    for back in (False, True):
        yq, yk = (ea.rope_bwd if back else ea.rope_fwd)(plan, q, k)
        check(yq, ref.rope(q.double(), pos, f, amp, inter, back), q, dim, inter, amp)
        check(yk, ref.rope(k.double(), pos, f, amp, inter, back), k, dim, inter, amp)
    only = ea.rope_fwd(plan, q)
    assert torch.equal(only, ea.rope_fwd(plan, q, k)[0])


@pytest.mark.parametrize("kw", [dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
                                dict(scaling="yarn", factor=16.0, original_len=4096),
                                dict(scaling="yarn", factor=2.0, original_len=64, base=500000.0)])
def test_scaled_and_far_positions(kw):
    """Positions up to the end of int32, where an fp32 angle would be lost."""
    plan = ea.Rope(128, **kw)
    f, amp = ref.rope_freqs(128, kw.get("base", 10000.0), kw["scaling"], kw["factor"], kw.get("original_len"))
    pos = torch.tensor([0, 1, 4095, 131071, 2 ** 20 + 3, 2 ** 24 + 1, 2 ** 31 - 1, -1, -70000], device="cuda")
    q = rand((1, 9, 2, 128), torch.float32, 3)
    y = ea.rope_fwd(plan, q, positions=pos.to(torch.int32))
    # at 2^31 the reference's own angle (a double) is off by 2^31 * 2^-53 * 2: 5e-7
    want = ref.rope(q.double(), pos[None], f.cuda(), amp, False)
    near = [i for i in range(9) if i != 6]
    check(y[:, near], want[:, near], q[:, near], 128, False, amp)
    assert (y[:, 6].double() - want[:, 6]).abs().max() < 3e-6 * q.abs().max().item() * amp


@pytest.mark.parametrize("lens", [[1], [5, 0, 1, 300, 17], [0, 0, 3], [129, 64]])
def test_packed(lens):
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    T = sum(lens)
    both = rand((T + 3, 6, 64), torch.bfloat16, 4)  # slices of one projection, rows behind the last sequence
    q, k = both[:, :4], both[:, 4:]
    plan = ea.Rope(64, interleaved=True)
    f, amp = ref.rope_freqs(64)
    out = (torch.full_like(q, 7.0).contiguous(), torch.full_like(k, 7.0).contiguous())
    yq, yk = ea.rope_fwd(plan, q, k, cu_seqlens=cu, out=out)
    pos = torch.cat([torch.arange(n) for n in lens]).cuda()
    check(yq[:T], ref.rope(q[:T].double(), pos, f.cuda(), amp, True), q[:T], 64, True, amp)
    check(yk[:T], ref.rope(k[:T].double(), pos, f.cuda(), amp, True), k[:T], 64, True, amp)
    assert (yq[T:] == 7).all() and (yk[T:] == 7).all()


def test_in_place_strides_and_positions():
    qkv = rand((2, 19, 3, 4, 128), torch.bfloat16, 5)  # [B, N, (q, k, v), H, d]
    keep = qkv.clone()
    pos = torch.randint(0, 10000, (2, 19), device="cuda", dtype=torch.int32)
    plan = ea.Rope(64)
    f, amp = ref.rope_freqs(64)
    q, k = qkv[:, :, 0], qkv[:, :, 1]
    ea.rope_fwd(plan, q, k, positions=pos.reshape(-1), out=(q, k))
    for i, x in ((0, q), (1, k)):
        check(x, ref.rope(keep[:, :, i].double(), pos, f.cuda(), amp, False), keep[:, :, i], 64, False, amp)
    assert torch.equal(qkv[:, :, 2], keep[:, :, 2])
    # heads outside tokens: [B, H, N, d] seen as [B, N, H, d]
    x = rand((2, 4, 19, 128), torch.float16, 6).transpose(1, 2)
    check(ea.rope_fwd(plan, x, positions=pos.reshape(-1)), ref.rope(x.double(), pos, f.cuda(), amp, False), x, 64, False, amp)


def test_gradient_against_differences():
    """<g, dF/dx v> by central differences of the forward (fp32) equals <bwd(g), v>.  The map is
    linear: differences are exact up to the fp32 roundings of the two sides (2^-22 of the norms)."""
    plan = ea.Rope(64, interleaved=True, scaling="yarn", factor=4.0, original_len=128)
    x, v, g = (rand((1, 50, 3, 128), torch.float32, s) for s in (7, 8, 9))
    h = 0.5
    num = (g.double() * (ea.rope_fwd(plan, x + h * v).double() - ea.rope_fwd(plan, x - h * v).double())).sum() / (2 * h)
    ana = (ea.rope_bwd(plan, g).double() * v.double()).sum()
    assert abs(num - ana) <= 2 ** -20 * g.double().norm() * v.double().norm()


def test_many_tokens_and_none():
    plan = ea.Rope(32)
    f, amp = ref.rope_freqs(32)
    x = rand((1, 100003, 1, 64), torch.bfloat16, 10)
    check(ea.rope_fwd(plan, x), ref.rope(x.double(), torch.arange(100003, device="cuda")[None], f.cuda(), amp, False), x, 32, False, amp)
    assert ea.rope_fwd(plan, x[:, :0]).shape == (1, 0, 1, 64)


def test_other_stream_and_graph():
    plan = ea.Rope(128)
    q, k = rand((2, 300, 4, 128), torch.bfloat16, 11), rand((2, 300, 2, 128), torch.bfloat16, 12)
    want = ea.rope_fwd(plan, q, k)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ea.rope_fwd(plan, q, k, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = ea.rope_fwd(plan, q, k)
    q.copy_(rand(q.shape, torch.bfloat16, 13))
    graph.replay()
    assert torch.equal(held[0], ea.rope_fwd(plan, q)) and torch.equal(held[1], want[1])
    ea.get_device_status()
