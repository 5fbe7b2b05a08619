"""What the paged-cache kernels' sources have to keep to, and refusals that the host decides."""
import os
import re

import pytest
import torch

from tests.test_paged_cpu import skv  # noqa: F401 (a fixture)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_kv_cache_gb300", "csrc")


def code_of(name):
    """A source without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_kernels_that_start_early_read_coherently():
    """The paged kernels are programmatic dependents: they are on the device while the kernels before them
    still write.  Loads of the non-coherent path are for data that nothing writes in a kernel's
    lifetime, and after the wait for those kernels only the other loads are sure to see it."""
    for name in ("skv_paged.h", "k_norm_rope.cu", "k_paged_attn.cu", "k_evict.cu"):
        assert not re.findall(r"\.nc\b|__ldg\b|__restrict__", code_of(name)), name
    # and the first kernel of a sparse decode step, which reads what the norm made
    head = re.search(r"k_qsplit\((.*?)\)", code_of("k_score.cu"), re.S).group(1)
    assert "__restrict__ q," not in head


@pytest.mark.parametrize("op,fields", [("attn", ("table", "lens", "lse", "weight", "weight_out")),
                                       ("evict", ("table", "lens", "lens_out")),
                                       ("norm", ("table", "positions", "seq", "index", "row_position", "row_weight"))])
def test_pointers_between_elements_are_refused(skv, op, fields):  # noqa: F811
    """Arrays of four-byte elements that begin between two of them."""
    from sparse_kv_cache_gb300 import _binding as b
    lib, host = skv.load(), torch.zeros(64)
    at = (host.data_ptr() + 15) & ~15
    names = ("table", "lens", "q", "lse", "weight", "weight_out", "position", "lens_out", "positions", "seq", "index",
             "row_position", "row_weight")

    def call(odd):
        a = {n: at + (2 if n == odd else 0) for n in names}
        cache = (1, 2, 128, 16, 1, 4, 8, 4096, 2048, 128, 4096, 2048, 128, 4, at, at, a["table"], a["lens"])
        if op == "attn":
            return lib.shadowkv_paged_attention(b._PAGED_ATTN.pack(
                *cache, 4, 0.0, 512, 128, 512, 128, at, at, a["lse"], a["weight"], a["weight_out"], 64, at, 1 << 40), None)
        if op == "evict":
            return lib.shadowkv_paged_evict(b._EVICT.pack(
                *cache, 8, 0, 0, at, at, at, at, 64, a["lens_out"], at, 1 << 40), None)
        return lib.shadowkv_qk_norm_rope(b._NORM_ROPE.pack(
            *cache, 1, 4, 0, 1e-6, 1e4, 512, 128, 256, 128, 256, 128, 512, 128, 256, 128, at, at, at, 0, 0, at, at,
            a["positions"], a["seq"], a["index"], a["row_position"], a["row_weight"], 64), None)

    # a good call gets as far as the look at the device (or at the memory, which is the host's)
    dev = lib.shadowkv_paged_status(None) == 0
    assert call(None) == (-1 if dev else -4)
    for odd in fields:
        assert call(odd) == -1, odd
