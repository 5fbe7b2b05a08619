"""The rules of test_paged_source.py for all files of the paged kernels, those that its list does not name among them."""
import os
import re

from tests.test_paged_source import CSRC, code_of


def test_all_kernels_that_start_early_read_coherently():
    names = [n for n in sorted(os.listdir(CSRC)) if n.endswith((".cu", ".cuh", ".h"))]
    early = [n for n in names if re.search(r"\bbegin_call\(\)|\bpdl_wait\(\)", code_of(n))
             and re.search(r'#include "(skv_paged\.h|paged_attn\.cuh)"', code_of(n))]
    assert {"paged_attn.cuh", "k_quantise.cu", "k_prompt_attn.cu", "k_norm_rope.cu"} <= set(early)
    for name in early + ["skv_paged.h"]:
        assert not re.findall(r"\.nc\b|__ldg\b|__restrict__", code_of(name)), name


def test_waits_of_the_paged_kernels_have_an_end():
    """Each wait for a barrier goes through a function with a limit."""
    for name in ("paged_attn.cuh", "k_prompt_attn.cu"):
        assert not re.findall(r"try_wait|mbar_wait\b", code_of(name)), name
