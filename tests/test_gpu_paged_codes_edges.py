"""Attention over codes where its kernels' forms end.  (Sizes and tolerances as in test_gpu_paged_codes.py.)"""
import os

import pytest
import torch

import sparse_kv_cache_gb300 as skv
from tests.test_gpu_paged_codes import Codes, ask, attend, check_codes

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
