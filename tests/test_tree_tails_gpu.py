"""Attention over the paged cache where one key takes most of a row's weight and many small ones
share the rest, against the definition in 64 bits.

Tolerance.  The scores are exact products (q and k meet in one value of the head; every number
is representable), so a weight is off by the fp32 arithmetic of its exponent (below 2e-6 * 20) and
the exponential: inside 2e-4 A, A = sum p |v|.  Probabilities: bf16, or for an E4M3 cache fp16 (2^-11) as
the sum of three E5M2 terms, whose last is off by 2^-9: below 2^-8 p either way; O is rounded to
bf16: 2^-8 |O|.  The E5M2 terms' smallest step is 2^-16, half of it 2^-17, and fp16's below its
normal numbers 2^-25; weights are stored times 2^11 relative to a reference that is never above the
row's final maximum, so that is an absolute 2^-28 (1 + 2^-8) F with F = sum |v| / sum exp(s - max).
Here F <= A exp(gap), whatever the number of keys: at the largest gap, 13, below 2^-9 A."""
import pytest
import torch

import exact_attention_103_b200 as ea
import serve_ref as ref

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def peaked(L, n, Hq, d, dtype, gap, at=0, page=64):
    """One sequence of L tokens: key `at` scores `gap`, every other between -0.25 and 0.25; values
    near 1 behind the small weights, 0 behind the large one."""
    g = torch.Generator(device="cuda").manual_seed(L + n)
    scale = 0.0625 if dtype == E4M3 else 1.0
    pages = -(-L // page)
    k, v = (torch.zeros(pages * page, 1, d, device="cuda") for _ in range(2))
    k[:L, 0, 0] = (torch.rand(L, generator=g, device="cuda") - 0.5) * 0.5
    v[:L, 0] = 0.5 + torch.rand(L, d, generator=g, device="cuda")
    k[at, 0, 0], v[at, 0] = gap, 0
    k, v = ((x / scale).to(dtype).view(1, pages, page, 1, d) for x in (k, v))
    c = ea.KVCache(k, v, ints([list(range(pages))]), ints([L]), ints([1] * pages), k_scale=scale, v_scale=scale)
    q = torch.randn((n, Hq, d), generator=g, device="cuda").to(torch.bfloat16)
    q[:, :, 0] = 1
    return c, q


# bf16 probabilities have no smallest step that matters: one gap shows it
CASES = [(E4M3, d, L, gap) for d in (128, 64) for L in (300, 4096, 131072) for gap in (6, 10, 11, 13)]
CASES += [(torch.bfloat16, 128, L, 13) for L in (300, 4096)]


@pytest.mark.parametrize("dtype,d,L,gap", CASES)
@pytest.mark.parametrize("n,G", [(1, 1), (1, 20), (10, 4), (25, 4), (50, 4)])
def test_one_key_over_a_flat_tail(dtype, d, n, G, L, gap):
    # the large key at the front, and behind thousands of small ones
    for at in (0, L // 2 + 5):
        c, q = peaked(L, n, G, d, dtype, gap, at)
        o, lse = ea.tree_fwd(c, q, ints([0, n]), scale=1.0)
        ea.get_device_status()
        row = c.page_table[0].tolist()
        k = ref.gather(c.k[0], row, L, c.page_size).double() * c.k_scale
        v = ref.gather(c.v[0], row, L, c.page_size).double() * c.v_scale
        seen = torch.ones(n, L, dtype=torch.bool, device="cuda")
        seen[:, L - n:] = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
        wo, wl, A, F = ref.attend(q, k, v, seen, 1.0)
        tol = 2 ** -8 * (A + wo.abs()) + 2e-4 * A + (2 ** -28 * 1.01 * F if dtype == E4M3 else 0)
        err = (o.double() - wo).abs()
        assert (err <= tol).all(), (at, (err / tol).max().item(), (err.norm() / wo.norm()).item())
        assert (lse.double().t() - wl).abs().max() <= 1e-4
