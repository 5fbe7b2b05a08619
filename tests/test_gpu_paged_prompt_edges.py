"""Prompts' attention where its kernels' forms end: heads that do not fill a tile, and what a caller may do that
test_gpu_paged_prompt.py does not.  (Sizes and tolerances as there.)"""
import os

import pytest
import torch

import sparse_kv_cache_gb300 as skv
from tests.paged_harness import Paged
from tests.test_gpu_paged_prompt import ask, attend, check_all, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("G", [3, 5, 6, 7])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tokens", [[23, 14], [700, 90]])
def test_the_same_bits_whatever_ran_before(G, d, tokens):
    """128 query rows are not a whole number of tokens: the rows left over hold nothing of an earlier call."""
    c = Paged("bf16", [800, 574], 2, d, 16, seed=G)
    other = Paged("bf16", [800, 574], 2, d, 16, seed=G + 1)
    q = ask(c, G, tokens)
    want = attend(c, q, tokens, window=300, sink=4)
    check_all(c, tokens, q, *want, 300, 4)
    for i in range(6):
        attend(other, ask(other, 8 - i % 2, tokens, i, 10.0 ** (i - 2)), tokens)      # queries of another size
        got = attend(c, q, tokens, window=300, sink=4)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("tensor", "qkv")
@pytest.mark.parametrize("G,d,lens,tokens", [
    (4, 128, [200], [20]),                    # a half to a CTA
    (4, 128, [256, 130], [200, 100]),         # two halves
    (2, 64, [3000, 140], [5, 3]),             # parts, of a half
    (3, 128, [2500], [300]),                  # parts, of two halves
])
def test_waits_that_run_out(G, d, lens, tokens, tensor):
    """Copies that bring less than a kernel waits for: after its limit the call ends, with NaN and its status, and the next one
    is as if there had been none."""
    c = Paged("bf16", lens, 2, d, 16, seed=31)
    q = ask(c, G, tokens)
    want = attend(c, q, tokens)
    check_all(c, tokens, q, *want)
    assert skv.paged_status() == 0
    os.environ["SHADOWKV_FAULT"] = "wait:" + tensor
    try:
        out, lse = attend(c, q, tokens)
    finally:
        del os.environ["SHADOWKV_FAULT"]
    assert skv.paged_status() == -6 and skv.paged_status() == 0
    assert out.isnan().all() and lse.isnan().all()
    got = attend(c, q, tokens)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and skv.paged_status() == 0


@pytest.mark.parametrize("lens,tokens", [([16, 16, 16], 100),                # whole units
                                         ([3000, 16, 16], 100),              # parts
                                         ([400] * 40, 9000)])                # many units
def test_starts_that_fall_behind_a_longer_sequence_are_reported(lens, tokens):
    """A search among starts passes over a sequence that begins behind a later one: it is reported all the same, and what the
    call leaves out is left as it was."""
    c = Paged("bf16", lens, 1, 64, 16, seed=5)
    q = ask(c, 2, [tokens])
    start = [0, tokens, 4, 8] + [8] * (len(lens) - 3)
    out = torch.full_like(q, 7.0)
    skv.paged_prompt_attention(q, c.k, c.v, c.table, c.lens, i32(start), out)
    assert skv.paged_status() == -5 and skv.paged_status() == 0
    # a bad length of a sequence without tokens
    start, bad = [0] + [tokens] * len(lens), i32(lens[:-1] + [-1])
    skv.paged_prompt_attention(q, c.k, c.v, c.table, bad, i32(start), out)
    assert skv.paged_status() == -5
    # rejected sequences' tokens are not touched
    for start in ([-3, tokens // 2, tokens + 1], [40, 0, 10], [0, tokens + 1, tokens + 2]):
        out.fill_(7.0)
        skv.paged_prompt_attention(q, c.k, c.v, c.table[:2], c.lens[:2], i32(start), out)
        assert skv.paged_status() == -5
        for t in range(tokens):
            of = [b for b in range(2) if 0 <= start[b] <= t < start[b + 1] <= tokens]
            if not of:
                assert (out[t] == 7).all()
