"""Prompts' attention where its kernels' forms end: heads that do not fill a tile, and what a caller may do that
test_gpu_paged_prompt.py does not.  (Sizes and tolerances as there.)"""
import math
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


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tokens", [3, 2500])
def test_sums_over_very_long_contexts(tokens, d):
    """16M rows, whole units of 2500 tokens and parts of units of 3.  What the tensor cores cut off of a sum, 2^-22 at every 16 rows, is that of
    131072 rows at most, 2^-9, however many there are; besides, as in test_gpu_paged_prompt.py, 2^-16 of the sums of
    probabilities (which are all alike, and exact) and 2^-8 of the result's rounding."""
    n, ps = 1 << 24, 1024
    k = torch.zeros((n // ps, 1, ps, d), dtype=torch.bfloat16, device="cuda")
    c = (1 + torch.arange(d, device="cuda") / 128).to(torch.bfloat16)      # exact
    v = c.expand(n // ps, 1, ps, d).contiguous()
    q = torch.ones((tokens, 8, d), dtype=torch.bfloat16, device="cuda")
    table = torch.randperm(n // ps, generator=torch.Generator().manual_seed(1)).to(torch.int32)[None].cuda()
    out, lse = torch.empty_like(q), torch.empty((tokens, 8), device="cuda")
    skv.paged_prompt_attention(q, k, v, table, i32([n]), i32([0, tokens]), out, lse)
    off = ((out.double() - c.double()) / c.double()).abs().max().item()
    assert off <= 2.0 ** -9 + 2.0 ** -16 + 2.0 ** -8, off
    want = torch.log(torch.arange(n - tokens + 1, n + 1, device="cuda").double())
    assert (lse.double() - want[:, None]).abs().max() <= 2.0 ** -16 + 2.0 ** -22 * math.log(n)
    assert skv.paged_status() == 0


@pytest.mark.parametrize("G,d,n,tokens,window,sink", [(8, 64, 600000, 2500, 0, 0), (2, 128, 300000, 20000, 200000, 300), (4, 128, 500000, 700, 0, 0)])
def test_long_contexts_match_float64(G, d, n, tokens, window, sink):
    ps = 64
    g = torch.Generator(device="cuda").manual_seed(n)
    k, v = (torch.randn((-(-n // ps), 1, ps, d), generator=g, device="cuda").bfloat16() for _ in range(2))
    v += 0.5
    q = torch.randn((tokens, G, d), generator=g, device="cuda").bfloat16()
    table = torch.randperm(k.shape[0], generator=g, device="cuda").to(torch.int32)[None]
    out, lse = torch.empty_like(q), torch.empty((tokens, G), device="cuda")
    skv.paged_prompt_attention(q, k, v, table, i32([n]), i32([0, tokens]), out, lse, window=window, sink=sink)
    rows = [x[table[0].long()].view(-1, d)[:n].double() for x in (k, v)]
    for t in (0, tokens // 2, tokens - 1):
        r, j = n - tokens + t, torch.arange(n, device="cuda")
        seen = (j <= r) & ((j > r - window) | (j < sink) if window else j >= 0)
        z = torch.where(seen, q[t].double() @ rows[0].T / math.sqrt(d), -math.inf)
        top = z.max(1, keepdim=True).values
        p = torch.exp(z - top)
        total = p.sum(1, keepdim=True)
        want, size = p / total @ rows[1], p / total @ rows[1].abs()
        delta = d * 2.0 ** -24 / math.sqrt(d) * (q[t].double().abs() @ rows[0].abs().T).max(1, keepdim=True).values
        tol = (2 * delta + 2.0 ** -8 + 2.0 ** -16 + min(n, 131072) * 2.0 ** -26) * size + 2.0 ** -8 * want.abs()
        assert ((out[t].double() - want).abs() <= tol).all()
        assert ((lse[t].double() - (top + torch.log(total))[:, 0]).abs() <= delta[:, 0] + 2.0 ** -16 + 2.0 ** -22 * 20).all()
    assert skv.paged_status() == 0


def test_very_long_contexts_on_two_streams_give_the_same_bits():
    n, ps, d, tokens = 400000, 64, 64, [2500, 4000]
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn((n // ps, 1, ps, d), generator=g, device="cuda").bfloat16() for _ in range(2))
    table, lens = torch.arange(n // ps, dtype=torch.int32, device="cuda")[None], i32([n])
    qs = [torch.randn((t, 8, d), generator=g, device="cuda").bfloat16() for t in tokens]
    starts = [i32([0, t]) for t in tokens]
    want = [skv.paged_prompt_attention(q, k, v, table, lens, s, torch.empty_like(q)) for q, s in zip(qs, starts)]
    streams = [torch.cuda.Stream() for _ in tokens]
    got = [[torch.empty_like(q) for _ in range(4)] for q in qs]
    torch.cuda.synchronize()
    for i in range(4):
        for j, st in enumerate(streams):
            skv.paged_prompt_attention(qs[j], k, v, table, lens, starts[j], got[j][i], stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(x, w) for x, w in zip(got[0] + got[1], [want[0]] * 4 + [want[1]] * 4))
    assert skv.paged_status() == 0


def test_handed_in_streams_give_the_same_bits():
    """Calls on two streams that were handed in, side by side: parts have a workspace of their own on each."""
    c = Paged("bf16", [5000, 500, 0, 3000], 2, 128, 16, seed=18)
    tokens = [[3, 200, 0, 1], [1, 1, 0, 7]]
    qs = [ask(c, 4, t, 19 + i) for i, t in enumerate(tokens)]
    starts = [i32([0, *torch.tensor(t).cumsum(0).tolist()]) for t in tokens]
    want = [attend(c, q, t) for q, t in zip(qs, tokens)]
    for q, t, w in zip(qs, tokens, want):
        check_all(c, t, q, *w)
    got = [[(torch.full_like(q, math.nan), torch.full(q.shape[:2], math.nan, device="cuda")) for _ in range(6)] for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for i in range(6):
        for j, s in enumerate(streams):
            skv.paged_prompt_attention(qs[j], c.k, c.v, c.table, c.lens, starts[j], *got[j][i], stream=s if i % 2 else s.cuda_stream)
    torch.cuda.synchronize()
    for j in range(2):
        assert all(torch.equal(o, want[j][0]) and torch.equal(s, want[j][1]) for o, s in got[j])
    assert skv.paged_status() == 0
