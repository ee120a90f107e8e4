"""Scaled frequencies of the rotary plans against the method's statement, written out here index by
index: YaRN keeps what turns more than beta_fast times over the trained length, divides by the factor
what turns less than beta_slow times, and goes linearly over the index between, from the floor of the one
border to the ceiling of the other, which may lie behind the last pair."""
import math

import pytest

import exact_attention_103_b200 as ea


@pytest.mark.parametrize("dim,base,L,factor", [
    (64, 10000.0, 131072, 8.0), (128, 10000.0, 65536, 4.0), (128, 10000.0, 4096, 16.0), (128, 500000.0, 8192, 8.0),
    (64, 500000.0, 1 << 20, 2.0), (32, 10000.0, 1 << 22, 32.0), (16, 10000.0, 64, 2.0), (16, 10000.0, 8, 2.0)])
def test_yarn(dim, base, L, factor):
    plan = ea.Rope(dim, base=base, scaling="yarn", factor=factor, original_len=L, device="cpu")
    got = [t / 2.0 ** 64 * 2 * math.pi for t in plan.turns.tolist()]

    def border(turns):  # the index whose frequency turns that often over L positions
        return dim * math.log(L / (turns * 2 * math.pi)) / (2 * math.log(base))
    first, last = max(math.floor(border(32.0)), 0), min(math.ceil(border(1.0)), dim - 1)
    for i, f in enumerate(got):
        plain = base ** (-2 * i / dim)
        part = min(max((i - first) / max(last - first, 1e-3), 0.0), 1.0)
        # 2^-48 relative for the doubles, half a unit of the fixed point absolutely
        assert f == pytest.approx(plain * (1 - part) + plain / factor * part, rel=2 ** -48, abs=2 ** -65 * 2 * math.pi)
        turns = L * plain / (2 * math.pi)
        if turns >= 32:
            assert f == pytest.approx(plain, rel=2 ** -48)
        if turns > 1 and i > 0:  # never the whole factor above one turn
            assert f > plain / factor * (1 + 1e-9)
    assert plan.amplitude == pytest.approx(0.1 * math.log(factor) + 1, rel=1e-15)
