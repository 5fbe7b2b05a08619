"""The paged-cache calls where sums are long, values extreme, pages bad or kernels of several calls
overlap.  Tolerances as derived in tests/test_gpu_paged.py, unless a test says otherwise."""
import math

import numpy as np
import pytest
import torch

import sparse_kv_cache_gb300 as skv
from oracle import paged_ref as ref
from tests.paged_harness import KINDS, Paged, f64
from tests.test_gpu_paged import U, UP, check_all, check_attention, check_norm, queries

pytestmark = pytest.mark.gpu


def wider(table, rows, ps):
    """The table with room for `rows` rows more of every sequence."""
    more = torch.full((table.shape[0], rows // ps), -1, dtype=torch.int32, device=table.device)
    return torch.cat([table, more], 1)


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


@pytest.mark.parametrize("headroom", [0, 16384])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "f32"])
def test_log_sum_exp_near_zero(kind, headroom):
    """Of one row it is the row's score, where the base lies: the rest is exp2 of a difference near 0 (off by
    2^-22 at most), its logarithm, and roundings of the result.  With e5m2 values the base lies 7 lower: two
    roundings of numbers near 7, 2^-22 each, and a logarithm near 7, 2^-21."""
    c = Paged(kind, [1] * 300, 1, 64, 16, seed=63)
    q = queries(c, 4, 64, 0.02)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    skv.paged_attention(q, c.k, c.v, wider(c.table, headroom, 16), c.lens, out, lse)
    for b in range(300):
        z = f64(q[b]) @ f64(c.krows[b][0, 0]) / 8
        delta = 64 * 2.0 ** -24 / 8 * (np.abs(f64(q[b])) @ np.abs(f64(c.krows[b][0, 0])))
        tol = delta + 2.0 ** -21 + (2.0 ** -20 if kind == "fp8" else 0)
        assert (np.abs(f64(lse[b]) - z) <= tol).all(), np.abs(f64(lse[b]) - z).max()


# ------------------------------------------------------------------ infinite and large values

def put_value(c, b, row, dim, x):
    page, off = int(c.table[b, row // c.ps]), row % c.ps
    if c.kind == "fp8":
        c.v.view(torch.uint8)[page, :, off, dim] = {math.inf: 0x7C, -math.inf: 0xFC}[x]
    else:
        c.v[page, :, off, dim] = x


@pytest.mark.parametrize("headroom", [0, 16384])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "f32"])
def test_infinite_values_in_rows_that_count(kind, headroom):
    """sum p_j v_j with v_j infinite and p_j > 0 is that infinity, whatever p_j; with both, NaN."""
    lens = [1, 40, 3000, 700]
    c = Paged(kind, lens, 2, 64, 16, seed=51)
    q = queries(c, 4, 52, 0.5)
    for b, n in enumerate(lens):
        for dim, rows, x in ((1, [0], math.inf), (2, [n - 1], -math.inf), (3, [n // 2, n // 3], math.inf)):
            for r in rows:
                put_value(c, b, r, dim, x)
        if n > 1:
            put_value(c, b, 0, 4, math.inf), put_value(c, b, n - 1, 4, -math.inf)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    skv.paged_attention(q, c.k, c.v, wider(c.table, headroom, 16), c.lens, out, lse)
    assert (out[..., 1] == math.inf).all() and (out[..., 2] == -math.inf).all() and (out[..., 3] == math.inf).all()
    assert out[1:, :, 4].isnan().all()
    # the other dimensions are what they are without
    out[..., 1:5] = 0
    for b in range(len(lens)):
        c.vrows[b][..., 1:5] = 0
    check_all(c, q, out, lse)


@pytest.mark.parametrize("headroom", [0, 16384])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_values_near_the_types_largest(kind, headroom):
    """The result lies between the values, so it is finite where they are: whatever the sums are before
    they are normalised.  Scores climb by less than the step at which a running base moves, and many rows
    share the weight."""
    lens = [5, 900, 20000]
    c = Paged(kind, lens, 1, 64, 16, seed=53)
    most = torch.finfo(KINDS[kind][0]).max
    for b, n in enumerate(lens):
        c.vrows[b][:, :, 0], c.vrows[b][:, :, 1] = 0.99 * most, -0.99 * most
        c.vrows[b][:, :, 2] = (torch.rand((1, n), generator=torch.Generator().manual_seed(n)) * most).to(c.v.dtype)
        c.krows[b].zero_()
        c.krows[b][:, 16:, 0] = 5.0                            # 2^7 above the first rows''
        for p in range(-(-n // 16)):
            hi = min(16, n - 16 * p)
            for pool, rows in ((c.k, c.krows), (c.v, c.vrows)):
                pool[int(c.table[b, p]), 0, :hi] = rows[b][0, 16 * p:16 * p + hi].cuda()
    q = torch.zeros((3, 2, 64), device="cuda").to(KINDS[kind][0])
    q[..., 0] = 1.0
    out, lse = torch.empty_like(q), torch.empty((3, 2), device="cuda")
    skv.paged_attention(q, c.k, c.v, wider(c.table, headroom, 16), c.lens, out, lse, scale=7 * math.log(2) / 5)
    assert out.isfinite().all()
    check_all(c, q, out, lse, 7 * math.log(2) / 5)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_small_values_keep_their_bits(kind):
    """Values near 2^-104 in a table for 16K rows: their products with 2^-22 of a probability lie near fp32's
    smallest normal number, 2^-126, and below it down to 2^-149: 2^-23 of that."""
    c = Paged(kind, [3000, 40], 1, 64, 16, seed=65)
    for b in range(2):
        c.vrows[b] = c.vrows[b] * 2.0 ** -104
    c.v = (c.v.float() * 2.0 ** -104).to(c.v.dtype)
    q = queries(c, 4, 66, 0.3)
    out = torch.empty_like(q)
    skv.paged_attention(q, c.k, c.v, wider(c.table, 13376, 16), c.lens, out)
    for b, n in enumerate(c.n):           # scaled up, with the tolerances of ordinary values
        check_attention(kind, f64(q[b]), f64(out[b]) * 2.0 ** 104, None, f64(c.krows[b][0]), f64(c.vrows[b][0]) * 2.0 ** 104, 0.125)


@pytest.mark.parametrize("headroom", [0, 16384])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_rows_that_a_negative_scale_brings_to_minus_infinity(kind, headroom):
    """Keys of +infinity under a negative scale score -infinity: such rows weigh nothing, one or all."""
    c = Paged(kind, [70, 50], 1, 64, 16, seed=54)
    q = queries(c, 2, 55).abs() + 0.5
    c.k[c.table[0, :5].long()] = math.inf
    c.k[int(c.table[1, 1]), 0, 3] = math.inf
    w = torch.rand((2, 1, c.rows + headroom), device="cuda")
    out, lse, got = torch.full_like(q, 9.0), torch.zeros((2, 2), device="cuda"), torch.zeros_like(w)
    skv.paged_attention(q, c.k, c.v, wider(c.table, headroom, 16), c.lens, out, lse, w, got, scale=-0.125)
    assert (out[0] == 0).all() and (lse[0] == -math.inf).all() and torch.equal(got[0, :, :70], w[0, :, :70])
    live = np.arange(50) != 19
    check_attention(kind, f64(q[1]), f64(out[1]), f64(lse[1]), f64(c.krows[1][0])[live], f64(c.vrows[1][0])[live], -0.125,
                    f64(w[1, 0, :50])[live], f64(got[1, 0, :50])[live])
    assert got[1, 0, 19] == w[1, 0, 19]


# ------------------------------------------------------------------ a CTA per unit with its products kept

@pytest.mark.parametrize("kind,G,d", [("bf16", 4, 128), ("bf16", 6, 128), ("bf16", 8, 128), ("fp8", 8, 128), ("bf16", 7, 64),
                                      ("f32", 8, 128), ("f32", 4, 64)])
def test_weights_of_as_many_units_as_fill_the_device(kind, G, d):
    """Rooms of 769 to 1024 rows, just as many units as CTAs: the most that a warp keeps in shared memory."""
    per = {"f32": 2}.get(kind, 3 if d == 128 else 4)
    units = torch.cuda.get_device_properties(0).multi_processor_count * per - 4
    c = Paged(kind, [1024 - (i * 37) % 300 for i in range(units // 4)], 4, d, 16, seed=56)
    q = queries(c, G, 57)
    w = torch.rand((units // 4, 4, c.rows), device="cuda")
    out, lse, got = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda"), torch.full_like(w, -7.0)
    skv.paged_attention(q, c.k, c.v, c.table, c.lens, out, lse, w, got)
    check_all(c, q, out, lse, None, w, got)
    for b, n in enumerate(c.n):
        assert (got[b, :, n:] == -7.0).all()


# ------------------------------------------------------------------ bad pages in an eviction

@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("budget,n", [(32, 64), (700, 1500)])          # moved by the search's own CTAs, by a second kernel
def test_a_row_that_cannot_move_leaves_the_place_as_it_was(budget, n, in_place):
    """A kept row in a bad page, or one whose new place is in one: key, value, weight and position of the
    place all stay those of the row that was given up there."""
    c = Paged("bf16", [n, n], 2, 64, 16, seed=58)
    g = torch.Generator().manual_seed(59)
    weight = torch.rand((2, 2, c.rows), generator=g).cuda()
    position = torch.stack([torch.randperm(c.rows, generator=g) for _ in range(4)]).view(2, 2, -1).to(torch.int32).cuda()
    good = c.table.clone()
    c.table[0, -1], c.table[1, 1] = c.k.shape[0] + 3, -2          # the last page; a page below the budget
    want_k, want_v, want_w, want_p = (x.clone().cpu() for x in (c.k, c.v, weight, position))
    if not in_place:
        want_w[:, :, budget:], want_p[:, :, budget:] = -3, -3
    t, stuck = good.cpu(), 0
    for b in range(2):
        for h in range(2):
            kept = ref.kept_rows(f64(weight[b, h, :n]), position[b, h, :n].cpu().numpy(), budget, 0, 0)
            for to, of in ref.moves(kept, budget):
                if of // 16 == c.table.shape[1] - 1 if b == 0 else to // 16 == 1:
                    stuck += 1
                    continue
                want_w[b, h, to], want_p[b, h, to] = weight[b, h, of].cpu(), position[b, h, of].cpu()
                for pool in (want_k, want_v):
                    pool[int(t[b, to // 16]), h, to % 16] = pool[int(t[b, of // 16]), h, of % 16]
    assert stuck > 4
    outs = {} if in_place else dict(weight_out=torch.full_like(weight, -3), position_out=torch.full_like(position, -3),
                                    lens_out=torch.empty_like(c.lens))
    skv.paged_evict(c.k, c.v, c.table, c.lens, weight, position, budget, **outs)
    assert skv.paged_status() == -5
    assert torch.equal(c.k.cpu().view(torch.int16), want_k.view(torch.int16))
    assert torch.equal(c.v.cpu().view(torch.int16), want_v.view(torch.int16))
    assert torch.equal(outs.get("weight_out", weight).cpu(), want_w)
    assert torch.equal(outs.get("position_out", position).cpu(), want_p)


# ------------------------------------------------------------------ errors of several streams

def test_no_error_is_lost_between_streams():
    """Bad calls on one stream while another's status is read all the time: every one is reported."""
    c = Paged("bf16", [64], 1, 64, 16, seed=60)
    q, bad = queries(c, 1), c.table.clone()
    bad[0, 2] = -1
    out = torch.empty_like(q)
    side, main = torch.cuda.Stream(), torch.cuda.Stream()
    skv.paged_attention(q, c.k, c.v, bad, c.lens, out)
    assert skv.paged_status() == -5
    for i in range(3000):
        seen, done = 0, torch.cuda.Event()
        with torch.cuda.stream(side):
            torch.cuda._sleep(2000 + i * 7919 % 160000)        # up to 80 us: a status takes 50
            skv.paged_attention(q, c.k, c.v, bad, c.lens, out, stream=side)
            done.record()
        over = False
        while not over:
            over = done.query()          # (asked before the status is: what is done then has to be in it)
            seen += skv.paged_status(main) != 0
        assert seen, f"call {i} was not reported"


# ------------------------------------------------------------------ dimensions that are not turned

@pytest.mark.parametrize("kind", ["bf16", "fp8", "f32"])
def test_dimensions_beyond_the_rotation_pass_through(kind):
    """Bit for bit where there is no norm, whatever their neighbours hold."""
    wide, g = KINDS[kind][0], torch.Generator().manual_seed(61)
    x = torch.randn((40, 3, 128), generator=g)
    pick = torch.rand(x.shape, generator=g)
    for lo, v in ((0.0, math.inf), (0.1, -math.inf), (0.2, 0.0), (0.3, -0.0), (0.4, 3e38)):
        x[(pick > lo) & (pick < lo + 0.1)] = v
    x[..., :64] = torch.randn((40, 3, 64), generator=g)
    x = x.to(wide).cuda()
    pos = torch.randint(0, 1 << 20, (40,), generator=g).to(torch.int32).cuda()
    c = Paged(kind, [0], 3, 128, 16, seed=62, cap=48)
    q_out, k_out = torch.empty_like(x), torch.empty_like(x)
    at = torch.arange(40, dtype=torch.int32, device="cuda")
    skv.qk_norm_rope(x, x, pos, q_out, k_out, rotary_dim=64, v=x, k_cache=c.k, v_cache=c.v, table=c.table,
                     seq=torch.zeros_like(at), index=at)
    bits = lambda t: t[..., 64:].contiguous().view(torch.uint8)  # noqa: E731
    held = c.k[c.table[0, at.long() // 16].long(), :, at.long() % 16]
    for out in (q_out, k_out, held):
        assert torch.equal(bits(out), bits(x))
    check_norm(x[..., :64], None, pos.cpu(), q_out[..., :64], kind, 500000.0, 64, 1e-6)
