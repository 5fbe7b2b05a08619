"""Attention over codes where its kernels' forms end.  (Sizes and tolerances as in test_gpu_paged_codes.py.)"""
import os

import numpy as np
import pytest
import torch

import sparse_kv_cache_gb300 as skv
from tests.test_gpu_paged_codes import E4M3, Codes, ask, attend, check_codes, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tensor", "kv")
@pytest.mark.parametrize("d,ps,lens", [
    (128, 16, [300]),                         # a cluster for a unit
    (64, 8, [5, 130, 0, 128] * 40),           # a CTA for a unit
    (128, 64, [20000, 3, 0, 7000]),           # parts of units, joined
    (64, 32, [900] * 30 + [30000]),           # several units to a warp
])
def test_waits_that_run_out(d, ps, lens, tensor):
    """Copies that bring less than a kernel waits for: after its limit the call ends, with NaN and its status, and the next one
    is as if there had been none."""
    c = Codes(lens, 2, d, ps, 8, seed=17)
    q = ask(c, 4)
    want = attend(c, q)
    check_codes(c, q, *want)
    assert skv.paged_status() == 0
    os.environ["SHADOWKV_FAULT"] = "wait:" + tensor
    try:
        out, lse = attend(c, q)
    finally:
        del os.environ["SHADOWKV_FAULT"]
    assert skv.paged_status() == -6 and skv.paged_status() == 0
    some = torch.tensor([n > 0 for n in lens])
    assert out[some].isnan().all() and lse[some].isnan().all()
    assert (out[~some] == 0).all() and (lse[~some] == -torch.inf).all()
    got = attend(c, q)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and skv.paged_status() == 0


@pytest.mark.parametrize("start", [[0, 100, 4, 8], [0, 100, 50, 50]])
def test_starts_that_fall_behind_a_longer_sequence_are_reported(start):
    """As for prompts: writing and reading back report a sequence that their searches pass over, and the rows of no good one
    are touched."""
    B, H, d, ps = 3, 2, 64, 16
    k = torch.randn((100, H, d), device="cuda")
    pools = [torch.full((30, H, ps, d), 0x55, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)]
    scales = [torch.full((30, H, 1), 3.0, device="cuda") for _ in range(2)]
    table = i32(np.arange(30).reshape(B, 10))
    skv.paged_quantise(k, k, *pools, *scales, table, i32([0] * B), i32(start))
    assert skv.paged_status() == -5 and skv.paged_status() == 0
    for pool, scale in zip(pools, scales):
        assert (pool[10:20].view(torch.uint8) == 0x55).all() and (scale[10:20] == 3).all()      # sequence 1 falls
    outs = [torch.full((100, H, d), 7.0, device="cuda") for _ in range(2)]
    skv.paged_dequantise(*pools, *scales, table, i32([100] * B), i32([0] * B), i32(start), *outs)
    assert skv.paged_status() == -5 and skv.paged_status() == 0
    # lengths and first rows of sequences without tokens
    for lens, first in (([100, -1, 100], [0, 0, 0]), ([100, 100, 1000], [0, 0, 0]), ([100, 100, 100], [0, -1, 0])):
        skv.paged_dequantise(*pools, *scales, table, i32(lens), i32(first), i32([0, 100, 100, 100]), *outs)
        assert skv.paged_status() == -5
        if min(first) == 0:
            skv.paged_quantise(k, k, *pools, *scales, table, i32([0] + lens[1:]), i32([0, 100, 100, 100]))
            assert skv.paged_status() == -5


@pytest.mark.parametrize("power,size", [(-96, 96), (-60, 60), (60, -60), (100, -100), (116, -100), (110, -90)])
def test_keys_far_from_one_and_queries_that_make_up_for_it(power, size):
    """Products of a code and a query, 2^32 at most, times a block's scale may be beyond fp32 where the score is not."""
    c = Codes([700, 45, 3], 2, 128, 16, 8, seed=23)
    c.ks.mul_(2.0 ** power)
    c.scales["k"] = [s * 2.0 ** power for s in c.scales["k"]]
    q = ask(c, 4, size=2.0 ** size)
    out, lse = attend(c, q)
    assert out.isfinite().all() and lse.isfinite().all()
    check_codes(c, q, out, lse)
