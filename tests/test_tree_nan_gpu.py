"""A score that is not a number makes its row's O and LSE not a number (an LSE of -inf would tell
whoever joins parts by LSE that the row saw nothing), in every form of the kernel, and no other
row's."""
import pytest
import torch

import exact_attention_103_b200 as ea
import test_tree_gpu as tree

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d", tree.KINDS)
@pytest.mark.parametrize("n,G", [(1, 4), (3, 8), (10, 4), (25, 4), (50, 4)])
@pytest.mark.parametrize("ctx", [[70, 260], [30000, 0]])
def test_query_that_is_not_a_number(dtype, d, n, G, ctx):
    c = tree.build(ctx, [n, n], 1, d, 64, dtype, seed=3)
    q, cu, o, lse = tree.run(c, [n, n], G)
    x = q.clone()
    x[n // 2, G - 1, 5] = float("nan")
    o2, lse2 = ea.tree_fwd(c, x, cu)
    ea.get_device_status()
    assert torch.isnan(o2[n // 2, G - 1]).all() and torch.isnan(lse2[G - 1, n // 2])
    o2[n // 2, G - 1], lse2[G - 1, n // 2] = o[n // 2, G - 1], lse[G - 1, n // 2]
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype,d", tree.KINDS)
@pytest.mark.parametrize("n,G", [(1, 4), (3, 8), (10, 4), (25, 4), (50, 4)])
@pytest.mark.parametrize("L,at", [(71, 3), (71, 70), (300, 140), (300, 299), (30000, 29999), (30000, 12345)])
@pytest.mark.parametrize("only", [False, True])
def test_key_that_is_not_a_number(dtype, d, n, G, L, at, only):
    """`only`: a mask leaves drafted rows one key of their own; the context's is what is NaN."""
    n = min(n, 40)
    L = max(L, n + 1)
    c = tree.build([L - n], [n], 1, d, 64, dtype, seed=4)
    at = min(at, L - n - 1) if not only else L - n  # the context is seen by all; or the first drafted token
    mask = torch.ones(n, n, dtype=torch.bool, device="cuda") if not only else torch.eye(n, dtype=torch.bool, device="cuda")
    q, cu, o, lse = tree.run(c, [n], G, mask)
    page = int(c.page_table[0, at // 64])
    c.k[0, page, at % 64, 0, 7] = float("nan")
    o2, lse2 = ea.tree_fwd(c, q, cu, mask=mask)
    ea.get_device_status()
    hit = mask[:, at - (L - n)] if at >= L - n else torch.ones(n, dtype=torch.bool, device="cuda")
    assert torch.isnan(o2[hit]).all() and torch.isnan(lse2[:, hit]).all()
    assert torch.equal(o2[~hit], o[~hit]) and torch.equal(lse2[:, ~hit], lse[:, ~hit])


@pytest.mark.parametrize("dtype", list(tree.SCALES))
def test_every_key_is_not_a_number(dtype):
    """No maximum to speak of in any part of a long context."""
    c = tree.build([20000], [2], 1, 128, 64, dtype, seed=4)
    q, cu, o, lse = tree.run(c, [2], 4)
    x = q.clone()
    x[0] = float("nan")
    o2, lse2 = ea.tree_fwd(c, x, cu)
    assert torch.isnan(o2[0]).all() and torch.isnan(lse2[:, 0]).all()
    assert torch.equal(o2[1], o[1]) and torch.equal(lse2[:, 1], lse[:, 1])
