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
