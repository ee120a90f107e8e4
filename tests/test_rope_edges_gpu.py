"""Calls of the rotary operators at the edge of what they document."""
import pytest
import torch

import exact_attention_103_b200 as ea
import serve_ref as ref
import test_rope_gpu as rope
import test_tree_gpu as tree

pytestmark = pytest.mark.gpu
ints = tree.ints


def test_packed_without_a_sequence():
    """Positions given: every packed row turns, also where cu_seqlens names no sequence at all."""
    plan = ea.Rope(64)
    f, amp = ref.rope_freqs(64)
    x = rope.rand((5, 2, 64), torch.bfloat16, 1)
    pos = torch.arange(3, 8, device="cuda", dtype=torch.int32)
    y = ea.rope_fwd(plan, x, positions=pos, cu_seqlens=ints([0]), out=torch.full_like(x, 7.0))
    rope.check(y, ref.rope(x.double(), pos, f.cuda(), amp, False), x, 64, False, amp)
    y = ea.rope_fwd(plan, x, cu_seqlens=ints([0]), out=torch.full_like(x, 7.0))
    assert (y == 7).all()


def test_strides_of_single_tokens_and_heads():
    """What a dimension of one element has as its stride is never used."""
    plan = ea.Rope(64)
    f, amp = ref.rope_freqs(64)
    flat = rope.rand((5000,), torch.bfloat16, 2)
    for shape, stride in (((1, 3, 64), (1111, 64, 1)), ((4, 1, 64), (64, 3, 1)), ((1, 1, 64), (5, 7, 1))):
        x = flat.as_strided(shape, stride)
        pos = torch.arange(9, 9 + shape[0], device="cuda", dtype=torch.int32)
        y = ea.rope_fwd(plan, x, positions=pos, cu_seqlens=ints([0, shape[0]]))
        rope.check(y, ref.rope(x.double(), pos, f.cuda(), amp, False), x, 64, False, amp)
        dense = flat.as_strided((1, *shape), (13, *stride))
        y = ea.rope_fwd(plan, dense, positions=pos)
        rope.check(y[0], ref.rope(x.double(), pos, f.cuda(), amp, False), x, 64, False, amp)
    c = tree.build([9], [1], 1, 64, 16)
    x = flat.as_strided((1, 1, 64), (5, 7, 1))
    ea.rope_append(c, None, x, x, ints([0, 1]))
    assert torch.equal(c.v[0, int(c.page_table[0, 0]), 9, 0], x[0, 0])
    with pytest.raises(ea.AttnError):
        ea.rope_fwd(plan, flat.as_strided((2, 1, 64), (68, 64, 1)), cu_seqlens=ints([0, 2]))
    ea.get_device_status()
