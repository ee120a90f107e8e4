"""Calls on a stream that is not the caller's: what a call allocates must not be memory that work queued
on the caller's stream still uses."""
import pytest
import torch

import exact_attention_103_b200 as ea
import test_tree_gpu as tree

pytestmark = pytest.mark.gpu
ints = tree.ints


def test_workspaces_of_two_streams():
    """A long call on the caller's stream, then at once one on another: the first one's workspace is free for
    its own stream only."""
    side = torch.cuda.Stream()
    a = tree.build([60000, 40000], [16, 16], 2, 128, 64, seed=1)
    b = tree.build([9000, 30000, 500], [7, 7, 7], 2, 128, 64, seed=2)
    g = torch.Generator(device="cuda").manual_seed(3)
    qa, qb = (torch.randn((t, 8, 128), generator=g, device="cuda").to(torch.bfloat16) for t in (32, 21))
    ca, cb = ints([0, 16, 32]), ints([0, 7, 14, 21])
    want_a, want_b = ea.tree_fwd(a, qa, ca), ea.tree_fwd(b, qb, cb)
    torch.cuda.synchronize()
    got = []
    for _ in range(30):
        side.wait_stream(torch.cuda.current_stream())
        got.append((ea.tree_fwd(a, qa, ca), ea.tree_fwd(b, qb, cb, stream=side)))
    torch.cuda.synchronize()
    for x, y in got:
        assert all(torch.equal(u, w) for u, w in zip(x + y, want_a + want_b))
    ea.get_device_status()


def test_memory_of_the_callers_stream():
    """Blocks freed on the caller's stream while a kernel there is yet to write them."""
    plan = ea.Rope(128)
    side = torch.cuda.Stream()
    q = torch.randn(1, 2048, 8, 128, device="cuda").to(torch.bfloat16)
    k = torch.randn(1, 2048, 8, 128, device="cuda").to(torch.bfloat16)
    c = tree.build([100, 50], [4, 4], 8, 128, 16, seed=4)
    ct = ints([0, 4, 8])
    qt = q[0, :8].contiguous()
    slots, lens = ints([0, 1]), c.lens.clone()
    calls = {
        "rope": lambda s: ea.rope_fwd(plan, q, k, stream=s),
        "append": lambda s: (ea.rope_append(c, qt, qt, qt, ct, plan=plan, stream=s),),
        "tree": lambda s: ea.tree_fwd(c, qt, ct, stream=s),
        "alloc": lambda s: (c.alloc(slots, lens, stream=s),),
    }
    busy = torch.randn(6000, 6000, device="cuda")
    for name, call in calls.items():
        want = [x.clone() for x in call(None)]
        torch.cuda.synchronize()
        for _ in range(3):
            (busy @ busy).sum()
            late = [torch.zeros_like(x) for x in want]  # written behind the product
            del late
            got = call(side)
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(got, want)), name
    ea.get_device_status()


def test_results_read_on_the_callers_stream():
    """A result dropped while the caller's stream is yet to read it is not handed to the next call."""
    plan = ea.Rope(128)
    side = torch.cuda.Stream()
    q = torch.randn(1, 4096, 8, 128, device="cuda").to(torch.bfloat16)
    p = -q
    want, other = ea.rope_fwd(plan, q), ea.rope_fwd(plan, p)
    busy = torch.randn(6000, 6000, device="cuda")
    torch.cuda.synchronize()
    for _ in range(3):
        y = ea.rope_fwd(plan, q, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        (busy @ busy).sum()
        z = y.clone()
        del y
        w = ea.rope_fwd(plan, p, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(z, want) and torch.equal(w, other)
    ea.get_device_status()


def test_forward_and_backward():
    """The dense calls: outputs, gradients and the backward's workspace."""
    side = torch.cuda.Stream()
    q, k, v, do = (torch.randn(1, 2048, 8, 128, device="cuda").to(torch.bfloat16) for _ in range(4))
    want = ea.fwd(q, k, v, causal=True)
    grads = ea.bwd(q, k, v, *want, do, causal=True)
    busy = torch.randn(6000, 6000, device="cuda")
    torch.cuda.synchronize()
    for _ in range(5):
        (busy @ busy).sum()
        late = [torch.zeros_like(x) for x in (*want, *grads)]  # written behind the product
        del late
        got = ea.fwd(q, k, v, causal=True, stream=side)
        back = ea.bwd(q, k, v, *want, do, causal=True, stream=side)
        over = [torch.full_like(q, 3.0) for _ in range(6)]  # what the backward released, if it could
        torch.cuda.synchronize()
        del over
        assert all(torch.equal(x, y) for x, y in zip((*got, *back), (*want, *grads)))
    ea.get_device_status()
