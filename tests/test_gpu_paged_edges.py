"""The paged-cache calls where sums are long, values extreme, pages bad or kernels of several calls
overlap.  Tolerances as derived in tests/test_gpu_paged.py, unless a test says otherwise."""
import math

import numpy as np
import pytest
import torch

import sparse_kv_cache_gb300 as skv
from oracle import paged_ref as ref
from tests.paged_harness import KINDS, f64
from tests.test_gpu_paged import U, UP

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ long sums

@pytest.mark.parametrize("flavour", ["spread", "equal"])
@pytest.mark.parametrize("kind,d,units", [("bf16", 128, 1900), ("bf16", 64, 2500), ("fp8", 128, 1900), ("f32", 64, 1900)])
def test_one_warp_walks_a_long_unit(kind, d, units, flavour):
    """So many sequences of 128K rows that a warp takes thousands of tiles of one by itself.  They share
    their pages.  Values of the first half are 1, of the second -1: what the sums lose on the way up does
    not come back on the way down."""
    n, ps, g = 1 << 17, 1024, torch.Generator().manual_seed(50)
    wide, val = KINDS[kind]
    k = torch.zeros((n, d)) if flavour == "equal" else torch.randn((n, d), generator=g)
    if flavour == "equal":
        k[0, 0] = 3.0                        # one score above all others, which are equal
    k = k.to(wide)
    v = torch.ones((n, d))
    v[n // 2:] = -1.0
    q = torch.randn((4, 1, d), generator=g) * 0.01 if flavour == "spread" else torch.zeros((4, 1, d))
    if flavour == "equal":
        q[:, 0, 0] = torch.tensor([0.25, 0.5, 0.75, 0.0])
    q = q.to(wide)
    pools = [x.view(n // ps, 1, ps, d).cuda() for x in (k, v.to(val))]
    table = torch.arange(n // ps, dtype=torch.int32, device="cuda").repeat(units, 1)
    lens = torch.full((units,), n, dtype=torch.int32, device="cuda")
    qs = q.cuda().repeat(units // 4, 1, 1)
    out, lse = torch.empty_like(qs), torch.empty((units, 1), device="cuda")
    scale = 1.0 if flavour == "equal" else 1 / math.sqrt(d)
    skv.paged_attention(qs, *pools, table, lens, out, lse, scale=scale)
    got, got_lse = f64(out), f64(lse)
    for i in range(4):
        want, want_lse, p = ref.attend(f64(q[i]), f64(k), f64(v), scale)
        delta = (d * 2.0 ** -24 * scale * (np.abs(f64(q[i])) @ np.abs(f64(k)).T)).max()
        tol = (2 * delta + UP[kind] + 2.0 ** -16) * (p @ np.abs(f64(v))) + U[kind] * np.abs(want) + 2.0 ** -32 * n
        bad = np.abs(got[i::4] - want) - tol
        assert (bad <= 0).all(), f"off by {np.abs(got[i::4] - want).max():.3g}, allowed {tol.min():.3g}"
        bad = np.abs(got_lse[i::4] - want_lse)
        assert (bad <= delta + 2.0 ** -16 + 2.0 ** -22 * np.abs(want_lse)).all(), f"lse off by {bad.max():.3g}"
    assert skv.paged_status() == 0
