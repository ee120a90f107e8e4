"""The serving operators' kernels are launched before the kernel in front of them has ended.  Loads by the
read-only path are only defined for memory that nobody writes while the kernel runs, from its launch on, so they
read nothing that way."""
import pathlib
import re

import pytest

CSRC = pathlib.Path(__file__).parents[1] / "exact_attention_103_b200" / "csrc"


@pytest.mark.parametrize("name", ["attn_tree_sm100.cu", "rope_sm100.cu", "cache_pages.cu", "cache_ops.h", "cache_ptx.cuh"])
def test_no_load_by_the_read_only_path(name):
    source = re.sub(r"//[^\n]*", "", (CSRC / name).read_text())
    assert not re.search(r"__ldg\b|ld\.global\.nc|ld\.global\.L\w+::\w+\.nc", source)
