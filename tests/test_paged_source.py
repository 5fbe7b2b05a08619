"""What the paged-cache kernels' sources have to keep to."""
import os
import re

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
