"""The paged-cache calls on the GPU against float64 forms of their definitions.

Tolerances, derived from the arithmetic (u = finfo.eps / 2 of the output type):

* norm and rotation: an fp32 sum of squares by a tree, rsqrt, two products, and a rotation whose
  cos and sin are within 2^-22.4 + 2^-23: below 2^-19 of the pair's length (of the element, where
  it passes through) in all, and one rounding: u |y|.
* attention: a score is an fp32 sum of d products, off by at most delta = d 2^-24 scale sum|q_i k_i|
  (any order); every probability then by 2 delta relatively (itself and the sum), and by u_p where it is
  rounded for the product with the values (two bf16 terms 2^-16, fp16 2^-11, fp32 0).  exp2 and the fp32 sums
  add less than 2^-16.  So |out - ref| <= (2 delta + u_p + 2^-16) sum p|v| + u |ref|; an fp16
  probability below the smallest normal one is off by 2^-25 against a top of 2^7 at least: 2^-32 sum|v|.
* lse: delta + 2^-16 + 2^-22 |lse|.   weights: G heads of p (2 delta + 2^-16), one fp32 sum.
* eviction copies: exact.
"""
import math

import numpy as np
import pytest
import torch

import sparse_kv_cache_gb300 as skv
from oracle import paged_ref as ref
from tests.paged_harness import KINDS, Paged, f64

pytestmark = pytest.mark.gpu

U = {"bf16": 2.0 ** -8, "fp8": 2.0 ** -8, "f32": 2.0 ** -24}
UP = {"bf16": 2.0 ** -16, "fp8": 2.0 ** -11, "f32": 0.0}


def check_attention(kind, q, got, lse, krows, vrows, scale, weight=None, weight_out=None):
    """q [G][d] float64 over a unit's rows; got [G][d], lse [G]; weight arrays [n]."""
    d = q.shape[1]
    out, want_lse, p = ref.attend(q, krows, vrows, scale)
    n = len(krows)
    delta = (d * 2.0 ** -24 * abs(scale) * (np.abs(q) @ np.abs(krows).T)).max(1) if n else np.zeros(len(q))
    tol = (2 * delta[:, None] + UP[kind] + 2.0 ** -16) * (p @ np.abs(vrows)) + U[kind] * np.abs(out) + \
        2.0 ** -32 * np.abs(vrows).sum(0)[None]
    assert not np.isnan(got).any()
    bad = np.abs(got - out) - tol
    assert (bad <= 0).all(), f"off by {np.abs(got - out).max():.3g}, allowed {tol.flat[bad.argmax()]:.3g}"
    if lse is not None:
        if n == 0:
            assert np.all(lse == -np.inf)
        else:
            assert (np.abs(lse - want_lse) <= delta + 2.0 ** -16 + 2.0 ** -22 * np.abs(want_lse)).all()
    if weight is not None:
        add = p.sum(0)
        tol = (p * (2 * delta[:, None] + 2.0 ** -16)).sum(0) + 2.0 ** -23 * (np.abs(weight) + add)
        assert (np.abs(weight_out - weight - add) <= tol).all()


def check_all(c, q, out, lse, scale=None, weight=None, weight_out=None):
    G = q.shape[1] // c.heads
    scale = scale or 1 / math.sqrt(c.d)
    qf, of = f64(q), f64(out)
    lf = f64(lse) if lse is not None else None
    for b, n in enumerate(c.n):
        for h in range(c.heads):
            s = slice(h * G, (h + 1) * G)
            w = (f64(weight[b, h, :n]), f64(weight_out[b, h, :n])) if weight is not None else (None, None)
            check_attention(c.kind, qf[b, s], of[b, s], lf[b, s] if lf is not None else None, f64(c.krows[b][h]),
                            f64(c.vrows[b][h]), scale, *w)


def queries(c, G, seed=1, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((len(c.n), c.heads * G, c.d), generator=g) * scale).to(KINDS[c.kind][0]).cuda()


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("kind,G,heads,d,ps,layout,lens", [
    ("bf16", 4, 2, 128, 16, "hnd", [1]),
    ("bf16", 1, 1, 64, 8, "nhd", [8, 9, 15, 16, 17, 1]),
    ("bf16", 8, 2, 128, 8, "hnd", [63, 64, 65, 0, 127, 128, 129]),
    ("bf16", 3, 3, 128, 32, "nhd", [1000, 0, 0, 5, 333]),
    ("bf16", 7, 1, 64, 1024, "hnd", [2049, 1023]),
    ("bf16", 8, 1, 128, 16, "hnd", [8190]),
    ("f32", 3, 2, 128, 16, "hnd", [6000, 0, 17]),
    ("fp8", 4, 1, 128, 16, "hnd", [2000] * 30 + [0, 3]),
    ("bf16", 2, 2, 128, 64, "nhd", [40000, 1, 0, 700]),        # one sequence over most of the CTAs
    ("bf16", 5, 8, 128, 16, "hnd", [300] * 40 + [0] * 200),    # several units per CTA, idle sequences behind
    ("bf16", 4, 1, 64, 16, "hnd", [0] * 150 + [77] + [0] * 150 + [3000]),
    ("bf16", 1, 1, 64, 8, "hnd", [(i * 7919) % 41 for i in range(1000)]),      # eight sequences per thread of the search
    ("bf16", 2, 1, 64, 16, "nhd", [(i * 31) % 23 for i in range(5000)]),       # runs of more than 32 sequences
    ("fp8", 1, 2, 64, 16, "hnd", [0] * 4500 + [900] + [0] * 200 + [5] * 100 + [0] * 30),
    ("bf16", 8, 4, 128, 16, "hnd", [(i * 97) % 700 for i in range(150)]),      # more units than CTAs are held at once
    ("f32", 4, 2, 64, 8, "hnd", [(i * 97) % 200 for i in range(200)]),
    ("fp8", 4, 2, 128, 16, "hnd", [1, 0, 500, 64]),
    ("fp8", 8, 1, 64, 8, "nhd", [1300, 7]),
    ("fp8", 1, 4, 128, 256, "nhd", [20000]),
    ("f32", 1, 2, 64, 8, "hnd", [1, 0, 77]),
    ("f32", 2, 1, 128, 16, "nhd", [3000, 12]),
    ("f32", 4, 2, 64, 32, "hnd", [700, 64, 65]),
    ("f32", 8, 1, 128, 8, "hnd", [129, 5000]),
    ("f32", 6, 2, 128, 64, "nhd", [63, 0, 1]),
])
def test_attention_matches_float64(kind, G, heads, d, ps, layout, lens):
    c = Paged(kind, lens, heads, d, ps, layout, seed=len(lens) + G)
    q = queries(c, G)
    # a table with room for far longer sequences: steps of few short ones are then split another way
    wide = torch.cat([c.table, torch.full((len(lens), 16384 // ps), -1, dtype=torch.int32, device="cuda")], 1)
    for table in (c.table, wide):
        for weigh in (False, True):
            out = torch.full_like(q, float("nan"))
            lse = torch.full(q.shape[:2], float("nan"), device="cuda")
            if weigh:
                weight = torch.rand((len(lens), heads, table.shape[1] * ps), device="cuda")
                held = torch.full_like(weight, -7.0)
                skv.paged_attention(q, c.k, c.v, table, c.lens, out, lse, weight, held)
                check_all(c, q, out, lse, None, weight, held)
                for b, n in enumerate(lens):
                    assert (held[b, :, n:] == -7.0).all()               # rows behind are left as they were
            else:
                skv.paged_attention(q, c.k, c.v, table, c.lens, out, lse)
                check_all(c, q, out, lse)
    assert skv.paged_status() == 0


@pytest.mark.parametrize("kind", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("scale,qs", [(1.0, 1.0), (-0.3, 1.0), (0.088, 60.0), (1e-6, 1.0)])
def test_scales_and_peaked_scores(kind, scale, qs):
    c = Paged(kind, [513, 200], 2, 128, 16, seed=3)
    q = queries(c, 4, 5, qs)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    skv.paged_attention(q, c.k, c.v, c.table, c.lens, out, lse, scale=scale)
    check_all(c, q, out, lse, scale)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "f32"])
def test_scores_that_climb(kind):
    """Every row scores above all rows before it: the running base moves all the time."""
    c = Paged(kind, [2000], 1, 128, 16, seed=4)
    ramp = torch.linspace(0.01, 6.0, 2000)[:, None].to(torch.bfloat16)
    for i in range(2000):
        c.krows[0][0, i] = ramp[i].to(c.krows[0].dtype)
    for p in range(125):
        c.k[int(c.table[0, p]), 0] = c.krows[0][0, 16 * p:16 * (p + 1)].cuda()
    q = torch.ones((1, 2, 128), device="cuda").to(KINDS[kind][0])
    out, lse = torch.empty_like(q), torch.empty((1, 2), device="cuda")
    skv.paged_attention(q, c.k, c.v, c.table, c.lens, out, lse, scale=0.05)
    check_all(c, q, out, lse, 0.05)


def test_small_probabilities_of_many_rows_add_up():
    """One row at the top and 20000 rows 2^-20 below it, whose values carry the result (e5m2 values,
    fp16 probabilities)."""
    c = Paged("fp8", [20001], 1, 64, 64, seed=6)
    c.krows[0].zero_()
    c.krows[0][0, 0, 0] = 20.0
    c.vrows[0] = torch.full((1, 20001, 64), 4096.0).to(torch.float8_e5m2)
    c.vrows[0][0, 0] = torch.zeros(64).to(torch.float8_e5m2)
    for p in range(313):
        lo, hi = 64 * p, min(64 * (p + 1), 20001)
        c.k[int(c.table[0, p]), 0, :hi - lo] = c.krows[0][0, lo:hi].cuda()
        c.v.view(torch.uint8)[int(c.table[0, p]), 0, :hi - lo] = c.vrows[0][0, lo:hi].view(torch.uint8).cuda()
    q = torch.zeros((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    q[0, 0, 0] = 1.0
    out = torch.empty_like(q)
    skv.paged_attention(q, c.k, c.v, c.table, c.lens, out, scale=math.log(2.0))
    check_all(c, q, out, None, math.log(2.0))
    assert f64(out).min() > 70                                          # 20000 * 4096 / 2^20 = 78


@pytest.mark.parametrize("kind", ["bf16", "fp8", "f32"])
def test_infinities_and_nan_in_rows_that_count_propagate(kind):
    c = Paged(kind, [100, 100, 100], 1, 64, 16, seed=7)
    q = queries(c, 2, 8).abs() + 0.5                     # every component positive
    c.k[int(c.table[0, 1]), 0, 3] = float("nan")         # a key: the sequence's results are NaN
    c.v.view(torch.uint8 if kind == "fp8" else c.v.dtype)[int(c.table[1, 1]), 0, 3, 5] = 0x7E if kind == "fp8" else float("nan")
    c.k[int(c.table[2, 2]), 0, 1] = float("-inf")        # scores -inf: the row weighs nothing
    c.krows[2][0, 33] = float("-inf")
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    skv.paged_attention(q, c.k, c.v, c.table, c.lens, out, lse)
    assert out[0].isnan().all() and lse[0].isnan().all()
    assert out[1, :, 5].isnan().all() and not out[1, :, :5].isnan().any() and not out[1, :, 6:].isnan().any()
    k2, v2 = f64(c.krows[2][0]), f64(c.vrows[2][0])
    live = np.arange(100) != 33
    check_attention(kind, f64(q[2]), f64(out[2]), f64(lse[2]), k2[live], v2[live], 0.125)


def test_rows_that_all_score_minus_infinity_give_zeros():
    c = Paged("bf16", [70], 1, 64, 16, seed=9)
    c.k[:] = float("-inf")
    q = torch.ones((1, 4, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.rand((1, 1, c.rows), device="cuda")
    out, lse, got = torch.full_like(q, 9.0), torch.zeros((1, 4), device="cuda"), torch.zeros_like(w)
    skv.paged_attention(q, c.k, c.v, c.table, c.lens, out, lse, w, got)
    assert (out == 0).all() and (lse == float("-inf")).all() and torch.equal(got[..., :70], w[..., :70])


def test_strided_queries_and_results():
    c = Paged("bf16", [333, 20], 2, 128, 16, "nhd", seed=10)
    fused = torch.randn((2, 3, 16, 128), device="cuda").to(torch.bfloat16)
    q = fused[:, 1, 4:12]                                  # a slice of a fused projection
    wide = torch.full((2, 8, 160), float("nan"), dtype=torch.bfloat16, device="cuda")
    out = wide[..., 16:144]
    skv.paged_attention(q, c.k, c.v, c.table, c.lens, out)
    check_all(c, q, out, None)
    assert wide[..., :16].isnan().all() and wide[..., 144:].isnan().all()


def test_strides_of_dimensions_that_are_not_stepped_through():
    """One sequence, one KV head: their strides may be anything, a row of 129 elements too."""
    c = Paged("bf16", [30], 1, 64, 16, seed=44)
    odd = lambda t: t.as_strided(t.shape, (t.stride(0), 129, t.stride(2), 1))  # noqa: E731
    q = torch.randn((1, 1, 64), device="cuda").to(torch.bfloat16).as_strided((1, 1, 64), (77, 33, 1))
    out = torch.empty_like(q)
    skv.paged_attention(q, odd(c.k), odd(c.v), c.table[:, :2].as_strided((1, 2), (5, 1)), c.lens, out)
    check_all(c, q, out, None)


def test_pages_of_two_sequences_may_be_the_same():
    c = Paged("bf16", [48, 48], 2, 128, 16, seed=11)
    c.table[1] = c.table[0]
    c.krows[1], c.vrows[1] = c.krows[0], c.vrows[0]
    q = queries(c, 4, 12)
    w = torch.rand((2, 2, c.rows), device="cuda")
    before = w.clone()
    out = torch.empty_like(q)
    skv.paged_attention(q, c.k, c.v, c.table, c.lens, out, weight=w)     # the sums are each sequence's own
    check_all(c, q, out, None, None, before, w)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_pools_beyond_32_bit_offsets(kind):
    """Pages 2^25 elements apart: their offsets pass 2^31 elements."""
    n, d, ps, step = 100, 128, 16, 1 << 25
    c = Paged(kind, [n], 1, d, ps, seed=13)
    wide = KINDS[kind][0]
    big = [torch.empty(step * 80, dtype=wide, device="cuda").as_strided((80, 1, ps, d), (step, ps * d, d, 1)) for _ in range(2)]
    table = torch.tensor([[79, 3, 78, 70, 65, 77, 68]], dtype=torch.int32, device="cuda")
    for pool, rows in zip(big, (c.krows, c.vrows)):
        for p in range(7):
            hi = min(16, n - 16 * p)
            pool[int(table[0, p]), 0, :hi] = rows[0][0, 16 * p:16 * p + hi].cuda()
            pool[int(table[0, p]), 0, hi:] = float("nan")
    q = queries(c, 4, 14)
    out = torch.empty_like(q)
    skv.paged_attention(q, *big, table, c.lens, out)
    check_all(c, q, out, None)
    # the append writes there too, and an eviction moves rows from there
    k = torch.randn((1, 1, d), device="cuda").to(wide)
    at = torch.tensor([n], dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    skv.qk_norm_rope(k, k, zero, torch.empty_like(k), v=k, k_cache=big[0], v_cache=big[1], table=table, seq=zero, index=at)
    assert torch.equal(big[0][68, 0, 4], k[0, 0]) and torch.equal(big[1][68, 0, 4], k[0, 0])
    w = torch.zeros((1, 1, 112), device="cuda")
    w[0, 0, 100] = 1.0
    pos = torch.arange(112, dtype=torch.int32, device="cuda")[None, None].contiguous()
    lens = torch.tensor([101], dtype=torch.int32, device="cuda")
    skv.paged_evict(*big, table, lens, w, pos, budget=50)
    assert torch.equal(big[0][70, 0, 1], k[0, 0]) and torch.equal(big[1][70, 0, 1], k[0, 0])
    assert int(lens) == 50 and int(pos[0, 0, 49]) == 100 and skv.paged_status() == 0


def test_bad_pages_and_lengths_are_reported_and_not_followed():
    c = Paged("bf16", [64, 40], 1, 64, 16, seed=15)
    q = queries(c, 2, 16)
    out = torch.empty_like(q)
    c.table[0, 1], c.table[0, 3] = -5, c.k.shape[0]
    live = np.r_[0:16, 32:48]
    w = torch.rand((2, 1, c.rows), device="cuda")
    held = torch.zeros_like(w)
    skv.paged_attention(q, c.k, c.v, c.table, c.lens, out, weight=w, weight_out=held)
    check_attention("bf16", f64(q[0]), f64(out[0]), None, f64(c.krows[0][0])[live], f64(c.vrows[0][0])[live], 0.125)
    assert torch.equal(held[0, 0, 16:32], w[0, 0, 16:32])               # absent rows received nothing
    assert skv.paged_status() == -5 and skv.paged_status() == 0
    lens = torch.tensor([-3, c.rows + 1], dtype=torch.int32, device="cuda")
    ok = torch.zeros_like(c.table)
    pool = torch.zeros_like(c.k)
    skv.paged_attention(q, pool, pool, ok, lens, out)
    assert (out == 0).all() and skv.paged_status() == -5
    # the append: rows, sequences and pages out of range are left out
    k = torch.ones((5, 1, 64), dtype=torch.bfloat16, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ok[0, 1] = 99
    skv.qk_norm_rope(k, k, i32(0, 0, 0, 0, 0), torch.empty_like(k), v=k, k_cache=pool, v_cache=pool, table=ok,
                     seq=i32(0, 2, 0, 0, 1), index=i32(c.rows, 0, -1, 16, 5))
    assert skv.paged_status() == -5
    assert float(pool.sum()) == 64.0 and float(pool[0, 0, 5].sum()) == 64.0
    # eviction: the rows of a bad page stay where they are
    rows = torch.arange(c.rows, device="cuda").float()[None, None].repeat(2, 1, 1)
    ok[:] = -1
    before = pool.clone()
    skv.paged_evict(pool, pool, ok, i32(20, 5), rows, rows.int(), budget=8)
    assert torch.equal(pool, before) and skv.paged_status() == -5


def test_host_memory_is_refused():
    c = Paged("bf16", [16], 1, 64, 16, seed=17)
    q = queries(c, 1)
    for bad in (dict(q=q.cpu()), dict(k_cache=c.k.cpu()), dict(table=c.table.cpu()), dict(lens=c.lens.cpu()), dict(out=q.cpu())):
        args = dict(q=q, k_cache=c.k, v_cache=c.v, table=c.table, lens=c.lens, out=torch.empty_like(q))
        with pytest.raises(skv.ShadowKVError) as e:
            skv.paged_attention(**{**args, **bad})
        assert e.value.code == -1
    rows = torch.zeros((1, 1, 16), device="cuda")
    with pytest.raises(skv.ShadowKVError):
        skv.paged_evict(c.k, c.v, c.table, c.lens, rows, rows.int().cpu(), budget=4)
    with pytest.raises(skv.ShadowKVError):
        skv.qk_norm_rope(q, q, c.lens.cpu(), q, q)


def test_two_calls_at_once_and_on_other_streams():
    c = Paged("bf16", [9000, 500, 0, 3000], 2, 128, 16, seed=18)
    a, b = queries(c, 4, 19), queries(c, 4, 20)
    want = [skv.paged_attention(x, c.k, c.v, c.table, c.lens, torch.empty_like(x)).clone() for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty_like(a) for _ in range(6)] for _ in range(2)]
    for i in range(6):
        for j, x in enumerate((a, b)):
            skv.paged_attention(x, c.k, c.v, c.table, c.lens, outs[j][i], stream=streams[j])
    torch.cuda.synchronize()
    for j in range(2):
        for o in outs[j]:
            assert torch.equal(o, want[j])               # the same bits each time


def test_captured_calls_replay_with_new_lengths():
    c = Paged("bf16", [700, 64], 2, 128, 16, seed=21)
    q = queries(c, 4, 22)
    outs = [torch.empty_like(q) for _ in range(2)]
    w = torch.zeros((2, 2, c.rows), device="cuda")
    skv.paged_attention(q, c.k, c.v, c.table, c.lens, outs[0])
    graphs = []
    for o in outs:                                       # two graphs, replayed on two streams at once
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            skv.paged_attention(q, c.k, c.v, c.table, c.lens, o, **({} if graphs else dict(weight=w)))
        graphs.append(g)
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for lens in ([700, 64], [1, 0], [333, 17], [0, 0]):
        c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        torch.cuda.synchronize()
        for g, st in zip(graphs, s):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        c.n = lens
        keep = c.krows, c.vrows
        c.krows = [x[:, :n] for x, n in zip(c.krows, lens)]
        c.vrows = [x[:, :n] for x, n in zip(c.vrows, lens)]
        for o in outs:
            check_all(c, q, o, None)
        c.krows, c.vrows = keep
    # one per query head, sequence with rows and replay
    assert float(w.sum()) == pytest.approx(8 * (2 + 1 + 2), rel=1e-3)


def test_calls_of_two_host_threads():
    import threading
    c = Paged("bf16", [3000, 100], 2, 128, 16, seed=23)
    qs = [queries(c, 4, 24 + i) for i in range(2)]
    want = [skv.paged_attention(x, c.k, c.v, c.table, c.lens, torch.empty_like(x)).clone() for x in qs]
    torch.cuda.synchronize()
    got, failed = [[], []], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                got[i] = [skv.paged_attention(qs[i], c.k, c.v, c.table, c.lens, torch.empty_like(qs[i])) for _ in range(50)]
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001 (reported by the test)
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for i in range(2):
        assert len(got[i]) == 50 and all(torch.equal(o, want[i]) for o in got[i])


def test_calls_of_two_host_threads_on_one_stream():
    """Each call is several kernels around one workspace; the threads' kernels must not alternate."""
    import threading
    c = Paged("bf16", [30000, 9000], 2, 128, 16, seed=27)
    qs = [queries(c, 4, 28 + i) for i in range(3)]
    ws = [torch.zeros((2, 2, c.rows), device="cuda") for _ in qs]
    want = [(skv.paged_attention(x, c.k, c.v, c.table, c.lens, torch.empty_like(x), weight=w).clone(), w.clone())
            for x, w in zip(qs, ws)]
    got, failed = [[] for _ in qs], []

    def work(i):
        try:
            for _ in range(40):
                w = torch.zeros_like(ws[i])
                got[i].append((skv.paged_attention(qs[i], c.k, c.v, c.table, c.lens, torch.empty_like(qs[i]), weight=w), w))
        except Exception as e:  # noqa: BLE001 (reported by the test)
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(qs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for mine, (out, w) in zip(got, want):
        assert len(mine) == 40 and all(torch.equal(o, out) and torch.equal(x, w) for o, x in mine)


def test_first_calls_of_a_process_inside_a_capture():
    """Every call captured before any was made: nothing needs a set-up outside the capture."""
    code = """
import torch, sparse_kv_cache_gb300 as skv
torch.manual_seed(0)
dev = "cuda"
i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)
k, v = (torch.randn(40, 2, 16, 64, device=dev).bfloat16() for _ in range(2))
table = torch.arange(40, dtype=torch.int32, device=dev).view(1, 40)
q = torch.randn(1, 8, 64, device=dev).bfloat16(); qr = torch.empty_like(q); out = torch.empty_like(q)
kn = torch.randn(1, 2, 64, device=dev).bfloat16()
w = torch.rand(1, 2, 640, device=dev); pos = torch.arange(640, dtype=torch.int32, device=dev).expand(1, 2, 640).contiguous()
lens, at, zero = i32(601), i32(600), i32(0)
saved = [t.clone() for t in (k, v, w, pos, lens)]
def step():
    skv.qk_norm_rope(q, kn, at, qr, v=kn, k_cache=k, v_cache=v, table=table, seq=zero, index=at, position=pos, weight=w)
    skv.paged_attention(qr, k, v, table, lens, out, weight=w)
    skv.paged_evict(k, v, table, lens, w, pos, 512, 16, 4)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    step()
g.replay()
torch.cuda.synchronize()
first = [t.clone() for t in (out, k, v, w, pos, lens)]
for t, s in zip((k, v, w, pos, lens), saved): t.copy_(s)
step()
torch.cuda.synchronize()
assert int(lens) == 512 and all(torch.equal(a, b) for a, b in zip(first, (out, k, v, w, pos, lens)))
assert skv.paged_status() == 0
print("same")
"""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=200)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]


# ------------------------------------------------------------------ norm, rotation, append

def check_norm(x, w, pos, got, kind, base, rd, eps):
    x, got = f64(x), f64(got)
    w = None if w is None else f64(w)
    for t in range(x.shape[0]):
        for h in range(x.shape[1]):
            want = ref.norm_rope(x[t, h], int(pos[t]), w, eps, base, rd)
            lo, hi = want[:rd // 2], want[rd // 2:rd]
            size = np.abs(want)
            size[:rd // 2] = size[rd // 2:rd] = np.hypot(lo, hi)
            bad = np.abs(got[t, h] - want) - (U[kind] * np.abs(want) + 2.0 ** -19 * size)
            assert (bad <= 0).all(), (t, h, bad.max())


@pytest.mark.parametrize("kind,n,nq,nk,d,rd,ps,layout,norms", [
    ("bf16", 1, 1, 1, 128, 128, 16, "hnd", "qk"),
    ("bf16", 7, 32, 8, 128, 128, 16, "hnd", ""),
    ("bf16", 33, 5, 3, 64, 32, 8, "nhd", "q"),
    ("bf16", 50, 0, 2, 128, 16, 64, "hnd", "k"),
    ("fp8", 19, 4, 1, 128, 128, 32, "nhd", "qk"),
    ("fp8", 40, 2, 2, 64, 48, 16, "hnd", ""),
    ("f32", 21, 3, 1, 64, 64, 8, "nhd", "qk"),
    ("f32", 9, 40, 2, 128, 96, 16, "hnd", "k"),
])
def test_norm_rope_append(kind, n, nq, nk, d, rd, ps, layout, norms):
    c = Paged(kind, [0, 0, 0], nk, d, ps, layout, seed=n, cap=64)
    g = torch.Generator().manual_seed(n + 1)
    wide = KINDS[kind][0]
    fused = (torch.randn((n, (nq + 2 * nk) * d), generator=g) * 3).to(wide).cuda()
    q, k = fused[:, :nq * d].unflatten(1, (nq, d)) if nq else fused[:, :0].view(n, 0, d), \
        fused[:, nq * d:(nq + nk) * d].unflatten(1, (nk, d))
    v = fused[:, (nq + nk) * d:].unflatten(1, (nk, d))
    wt = lambda on: (1 + torch.rand(d, generator=g)).to(wide).cuda() if on else None  # noqa: E731
    qw, kw = wt("q" in norms), wt("k" in norms)
    pos = torch.randint(0, 1 << 20, (n,), generator=g).to(torch.int32)
    pos[0], pos[n // 2] = 2 ** 31 - 1, 0
    if n > 6:
        pos[3] = -1                                             # padding
    place = torch.randperm(3 * 64, generator=g)[:n]
    seq, index = (place // 64).to(torch.int32), (place % 64).to(torch.int32)
    if n > 6:
        seq[5] = -1                                             # computed, not kept
    q_out = torch.full((n, nq, d), 77.0, dtype=wide, device="cuda")
    k_out = torch.full((n, nk, d), 77.0, dtype=wide, device="cuda")
    rows = torch.full((3, nk, c.rows), -5, dtype=torch.int32, device="cuda")
    sums = torch.full((3, nk, c.rows), -5.0, device="cuda")
    before = c.k.clone(), c.v.clone()
    dev = [x.cuda() for x in (pos, seq, index)]
    skv.qk_norm_rope(q, k, dev[0], q_out, k_out, q_weight=qw, k_weight=kw, eps=1e-5, rope_base=10000.0, rotary_dim=rd,
                     v=v, k_cache=c.k, v_cache=c.v, table=c.table, seq=dev[1], index=dev[2], position=rows, weight=sums)
    assert skv.paged_status() == 0
    live = [t for t in range(n) if pos[t] >= 0]
    check_norm(q[live], qw, pos[live], q_out[live], kind, 10000.0, rd, 1e-5)
    check_norm(k[live], kw, pos[live], k_out[live], kind, 10000.0, rd, 1e-5)
    dead = [t for t in range(n) if pos[t] < 0]
    assert (q_out[dead] == 77).all() and (k_out[dead] == 77).all()
    want_k, want_v, want_p, want_s = *before, torch.full_like(rows, -5), torch.full_like(sums, -5)
    raw = lambda x: x.view(torch.uint8) if kind == "fp8" else x  # noqa: E731
    for t in live:
        if seq[t] < 0:
            continue
        page, off = int(c.table[seq[t], index[t] // ps]), int(index[t]) % ps
        want_k[page, :, off] = k_out[t]
        raw(want_v)[page, :, off] = raw(v[t].to(c.v.dtype))
        want_p[seq[t], :, index[t]] = pos[t].cuda()
        want_s[seq[t], :, index[t]] = 0
    bits = lambda x: x.contiguous().view(torch.uint8)  # noqa: E731
    assert torch.equal(bits(c.k), bits(want_k)) and torch.equal(bits(c.v), bits(want_v))   # and nothing else was touched
    assert torch.equal(rows, want_p) and torch.equal(sums, want_s)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "f32"])
def test_norm_rope_of_a_prompt(kind, d):
    """As many tokens as take the form with more CTAs per SM."""
    n, nq, nk, ps = 1003, 2, 1, 16
    c = Paged(kind, [0], nk, d, ps, seed=31, cap=n)
    g = torch.Generator().manual_seed(32)
    wide = KINDS[kind][0]
    q, k, v = ((torch.randn((n, h, d), generator=g) * 2).to(wide).cuda() for h in (nq, nk, nk))
    w = (1 + torch.rand(d, generator=g)).to(wide).cuda()
    pos = torch.arange(70000, 70000 + n, dtype=torch.int32)
    pos[500] = -1
    index = torch.randperm(n, generator=g).to(torch.int32)
    q_out, k_out = (torch.full_like(x, 77.0) for x in (q, k))
    skv.qk_norm_rope(q, k, pos.cuda(), q_out, k_out, q_weight=w, k_weight=w, eps=1e-5, rope_base=10000.0, rotary_dim=d - 32,
                     v=v, k_cache=c.k, v_cache=c.v, table=c.table, seq=torch.zeros(n, dtype=torch.int32, device="cuda"),
                     index=index.cuda())
    assert skv.paged_status() == 0
    live = [t for t in range(n) if t != 500]
    for x, out in ((q, q_out), (k, k_out)):
        assert (out[500] == 77).all()
        check_norm(x[live], w, pos[live], out[live], kind, 10000.0, d - 32, 1e-5)
    at = index.long()[live].cuda()
    page, off = c.table[0].long()[at // ps], at % ps
    assert torch.equal(c.k[page, :, off], k_out[live])
    raw = lambda x: x.contiguous().view(torch.uint8)  # noqa: E731
    assert torch.equal(raw(c.v[page, :, off] if kind != "fp8" else c.v.view(torch.uint8)[page, :, off]), raw(v[live].to(c.v.dtype)))


def test_norm_rope_in_place_and_without_a_cache():
    for kind in ("bf16", "f32"):
        x = torch.randn((300, 12, 128), device="cuda").to(KINDS[kind][0])
        q, k = x[:, :9], x[:, 9:]
        was = x.clone()
        pos = torch.arange(300, dtype=torch.int32, device="cuda") * 997
        w = torch.rand(128, device="cuda").to(x.dtype)
        skv.qk_norm_rope(q, k, pos, q, k, q_weight=w, k_weight=w)
        check_norm(was[:, :9], w, pos.cpu(), q, kind, 500000.0, 128, 1e-6)
        check_norm(was[:, 9:], w, pos.cpu(), k, kind, 500000.0, 128, 1e-6)


def test_e5m2_append_saturates():
    c = Paged("fp8", [0], 1, 64, 8, seed=1, cap=8)
    v = torch.full((1, 1, 64), 1e5, device="cuda").to(torch.bfloat16)
    v[..., ::2] *= -1
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    skv.qk_norm_rope(v, v, z, torch.empty_like(v), v=v, k_cache=c.k, v_cache=c.v, table=c.table, seq=z, index=z)
    got = c.v[int(c.table[0, 0]), 0, 0].float()
    assert torch.equal(got.abs(), torch.full((64,), 57344.0, device="cuda")) and (got[::2] < 0).all()


# ------------------------------------------------------------------ eviction

def run_evict(c, weight, position, budget, recent, sink, in_place):
    """Evicts and compares every unit with the float64 form; returns the new lengths."""
    B, H = len(c.n), c.heads
    raw = lambda x: x.view(torch.uint8) if c.kind == "fp8" else x  # noqa: E731
    want_k, want_v = c.k.clone().cpu(), raw(c.v).clone().cpu()
    want_w = (weight if in_place else torch.full_like(weight, -3)).clone().cpu()
    want_p = (position if in_place else torch.full_like(position, -3)).clone().cpu()
    wc, pc, t = weight.cpu(), position.cpu(), c.table.cpu()
    for b, n in enumerate(c.n):
        for h in range(H):
            kept = ref.kept_rows(wc[b, h, :n].double().numpy(), pc[b, h, :n].numpy(), budget, recent, sink)
            for i in np.flatnonzero(kept[:budget]):
                want_w[b, h, i], want_p[b, h, i] = wc[b, h, i], pc[b, h, i]
            for to, of in ref.moves(kept, budget):
                want_w[b, h, to], want_p[b, h, to] = wc[b, h, of], pc[b, h, of]
                for pool in (want_k, want_v):
                    pool[int(t[b, to // c.ps]), h, to % c.ps] = pool[int(t[b, of // c.ps]), h, of % c.ps]
    outs = {} if in_place else dict(weight_out=torch.full_like(weight, -3), position_out=torch.full_like(position, -3),
                                    lens_out=torch.full_like(c.lens, -3))
    skv.paged_evict(c.k, c.v, c.table, c.lens, weight, position, budget, recent, sink, **outs)
    assert skv.paged_status() == 0
    bits = lambda x: x.cpu().contiguous().view(torch.uint8)  # noqa: E731
    assert torch.equal(bits(outs.get("position_out", position)), bits(want_p))
    assert torch.equal(bits(outs.get("weight_out", weight)), bits(want_w))
    assert torch.equal(bits(c.k), bits(want_k)) and torch.equal(bits(raw(c.v)), bits(want_v))
    assert outs.get("lens_out", c.lens).tolist() == [min(n, budget) for n in c.n]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind,lens,heads,d,ps,layout,budget,recent,sink,flavour", [
    ("bf16", [1, 0, 2, 3], 2, 64, 8, "hnd", 1, 0, 0, "plain"),
    ("bf16", [33, 32, 31, 0], 3, 128, 16, "nhd", 32, 8, 4, "plain"),
    ("bf16", [1000, 2081, 64], 2, 128, 16, "hnd", 512, 32, 4, "plain"),
    ("bf16", [777, 300], 1, 64, 32, "hnd", 299, 100, 7, "ties"),
    ("bf16", [513], 2, 128, 16, "nhd", 256, 0, 0, "equal"),
    ("fp8", [900, 1], 2, 128, 16, "hnd", 100, 10, 0, "wild"),
    ("f32", [450, 451], 2, 64, 8, "nhd", 450, 450, 0, "wild"),
    ("bf16", [10000, 9], 1, 64, 64, "hnd", 2464, 32, 4, "ties"),      # two CTAs per unit
    ("bf16", [40000], 2, 64, 64, "hnd", 1000, 32, 4, "ties"),         # eight
    ("bf16", [70000, 65000], 1, 64, 1024, "nhd", 66000, 9, 2, "plain"),
    ("bf16", [(i * 53) % 300 for i in range(50)], 7, 64, 16, "hnd", 90, 8, 2, "ties"),      # many short units
    ("fp8", [3000 - i for i in range(80)], 4, 64, 32, "nhd", 1200, 30, 2, "wild"),          # many units, many rows that move
])
def test_eviction_matches(kind, lens, heads, d, ps, layout, budget, recent, sink, flavour, in_place):
    c = Paged(kind, lens, heads, d, ps, layout, seed=budget)
    g = torch.Generator().manual_seed(budget + 1)
    shape = (len(lens), heads, c.rows)
    weight = torch.randn(shape, generator=g).mul(2).exp()
    if flavour == "ties":
        weight = torch.randint(0, 4, shape, generator=g).float() * 0.25
    elif flavour == "equal":
        weight = torch.ones(shape)
    elif flavour == "wild":
        weight = torch.randn(shape, generator=g)
        pick = torch.rand(shape, generator=g)
        for lo, x in ((0.0, float("nan")), (0.1, float("inf")), (0.2, float("-inf")), (0.3, -0.0), (0.5, 0.0), (0.7, 1e-42)):
            weight[(pick > lo) & (pick < lo + 0.04)] = x
    position = torch.stack([torch.stack([torch.randperm(c.rows, generator=g) * 2 for _ in range(heads)]) for _ in lens])
    run_evict(c, weight.cuda(), position.to(torch.int32).cuda(), budget, recent, sink, in_place)


def test_eviction_of_slices_beyond_shared_memory():
    """One unit over eight CTAs of more rows each than their shared memory holds keys."""
    n, budget = 400000, 5000
    g = torch.Generator(device="cuda").manual_seed(3)
    pool = torch.randn((n // 32, 1, 32, 64), generator=g, device="cuda").to(torch.bfloat16)
    table = torch.arange(n // 32, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([n - 5], dtype=torch.int32, device="cuda")
    weight = torch.randint(0, 1 << 16, (1, 1, n), generator=g, device="cuda").float()
    pos = torch.arange(n, dtype=torch.int32, device="cuda")[None, None].contiguous()
    k, v = pool.clone(), pool.clone()
    w_out, p_out, l_out = torch.zeros_like(weight), torch.zeros_like(pos), torch.zeros_like(lens)
    skv.paged_evict(k, v, table, lens, weight, pos, budget, 16, 16, l_out, w_out, p_out)
    key = weight[0, 0, :n - 5].double()
    key[-16:] = key[:16] = 1e9
    kept = torch.zeros(n - 5, dtype=torch.bool, device="cuda")
    kept[key.sort(descending=True, stable=True).indices[:budget]] = True
    rows = torch.arange(budget, device="cuda")
    rows[~kept[:budget]] = kept.nonzero().flatten()[kept[:budget].sum():]
    assert torch.equal(p_out[0, 0, :budget].long(), rows) and torch.equal(w_out[0, 0, :budget], weight[0, 0, rows])
    assert torch.equal(k.view(-1, 64)[:budget], pool.view(-1, 64)[rows]) and torch.equal(k, v) and int(l_out) == budget


@pytest.mark.parametrize("where", ["front", "behind", "spread"])
def test_eviction_where_the_heavy_rows_crowd(where):
    """A small budget out of a long sequence, with the rows that can stay in one place: within the
    budget's own rows, in one warp's rows behind it, or everywhere; near-equal weights, so that
    most of the search happens in the lower bits."""
    n, budget = 20000, 700
    c = Paged("bf16", [n, 15], 1, 64, 64, seed=40)
    g = torch.Generator().manual_seed(41)
    weight = torch.rand((2, 1, c.rows), generator=g) * 1e-3
    at = {"front": torch.arange(0, 900), "behind": torch.arange(9000, 9900), "spread": torch.randperm(n, generator=g)[:900]}[where]
    weight[0, 0, at] = 1.0 + torch.randint(0, 200, (900,), generator=g) * 2.0 ** -20
    position = torch.arange(c.rows, dtype=torch.int32).expand(2, 1, -1).contiguous()
    run_evict(c, weight.cuda(), position.cuda(), budget, 0, 0, False)


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("kind", ["bf16", "fp8", "f32"])
def test_decode_steps_over_a_budget(kind):
    """Prompts and decode steps as a server runs them: norm, rotation and append; attention that
    adds up the rows' weights; eviction in place -- captured into one graph per step, against the
    float64 forms on the cache as it stood before each call."""
    H, G, d, ps, budget, prompt = 2, 4, 64, 8, 40, [44, 13, 30]
    B, wide = 3, KINDS[kind][0]
    c = Paged(kind, [0] * B, H, d, ps, seed=30, cap=64)
    g = torch.Generator().manual_seed(31)
    draw = lambda n, h: (torch.randn((n, h, d), generator=g) * 2).to(wide).cuda()  # noqa: E731
    w = (1 + torch.rand(d, generator=g)).to(wide).cuda()
    pos = torch.full((B, H, c.rows), -1, dtype=torch.int32, device="cuda")
    sums = torch.full((B, H, c.rows), float("nan"), device="cuda")
    at = torch.cat([torch.arange(n, dtype=torch.int32) for n in prompt]).cuda()
    seq = torch.cat([torch.full((n,), b, dtype=torch.int32) for b, n in enumerate(prompt)]).cuda()
    q, k, v = draw(sum(prompt), H * G), draw(sum(prompt), H), draw(sum(prompt), H)
    skv.qk_norm_rope(q, k, at, q, q_weight=w, k_weight=w, v=v, k_cache=c.k, v_cache=c.v, table=c.table, seq=seq, index=at,
                     position=pos, weight=sums)
    c.lens.copy_(torch.tensor(prompt))
    each = torch.arange(B, dtype=torch.int32, device="cuda")
    positions = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    q, k, v, out, lse = draw(B, H * G), draw(B, H), draw(B, H), draw(B, H * G), torch.empty((B, H * G), device="cuda")
    qr = torch.empty_like(q)
    index = torch.zeros_like(c.lens)

    def step():
        index.copy_(c.lens)
        skv.qk_norm_rope(q, k, positions, qr, q_weight=w, k_weight=w, v=v, k_cache=c.k, v_cache=c.v, table=c.table, seq=each,
                         index=index, position=pos, weight=sums)
        c.lens.add_(1)
        skv.paged_attention(qr, c.k, c.v, c.table, c.lens, out, lse, sums)

    def give_up():
        skv.paged_evict(c.k, c.v, c.table, c.lens, sums, pos, budget, recent=8, sink=2)

    step(), give_up()
    torch.cuda.synchronize()
    graphs = []
    for f in (step, give_up):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            f()
        graphs.append(gr)
    seen = [prompt[b] + 1 for b in range(B)]
    for i in range(12):
        positions.add_(1)
        for x in (q, k, v):
            x.copy_(draw(B, x.shape[1]))
        before = sums.clone()
        graphs[0].replay()
        lens = c.lens.tolist()
        check_norm(q, w, positions.cpu(), qr, kind, 500000.0, d, 1e-6)
        for b in range(B):
            seen[b] += 1
            for h in range(H):
                n, s = lens[b], slice(h * G, (h + 1) * G)
                assert int(pos[b, h, :n].max()) == seen[b] - 1 and len(set(pos[b, h, :n].tolist())) == n
                before[b, h, n - 1] = 0
                check_attention(kind, f64(qr[b, s]), f64(out[b, s]), f64(lse[b, s]), c.stored("k", b, h, n),
                                c.stored("v", b, h, n), 0.125, f64(before[b, h, :n]), f64(sums[b, h, :n]))
        c.n = lens
        # what the eviction keeps, by the float64 form on the sums as they stand
        want = [[ref.kept_rows(f64(sums[b, h, :n]), pos[b, h, :n].cpu().numpy(), budget, 8, 2) for h in range(H)]
                for b, n in enumerate(lens)]
        held = pos.clone()
        graphs[1].replay()
        assert c.lens.tolist() == [min(n, budget) for n in lens]
        for b in range(B):
            for h in range(H):
                keep = held[b, h, :lens[b]].cpu().numpy()[want[b][h]]
                assert sorted(pos[b, h, :min(lens[b], budget)].tolist()) == sorted(keep.tolist())
    assert c.lens.tolist() == [40, 26, 40] and skv.paged_status() == 0


def test_sparse_layer_takes_what_norm_rope_makes():
    """q and k_new of shadowkv_decode_step out of qk_norm_rope: the layer keeps that very key, and
    its output is the dense attention where its budget covers everything."""
    from tests.gpu_harness import LayerRun
    from workload import Workload
    w = Workload(name="paged-full-budget", layers=1, batch=1, seq_len=512, n_kv_heads=2, n_q_heads=8, head_dim=128, rank=160,
                 chunk=8, n_select=58, n_outlier=4, local_window=16, steps=2, dtype="bf16", v_place="hbm", drift=0.9, seed=5)
    run = LayerRun(w, 1)
    q, k, v = run.q_d[0], run.kn_d[0], run.vn_d[0]
    pos = torch.tensor([512], dtype=torch.int32, device="cuda")
    one = lambda x: x.view(1, -1, 128)  # noqa: E731
    qr, kr = skv.qk_norm_rope(one(q), one(k), pos, torch.empty_like(one(q)), torch.empty_like(one(k)), rope_base=w.rope_base)
    out = torch.empty_like(qr)
    torch.cuda.synchronize()
    run.layer.decode_step(qr, kr, v, out, main=run.main, side=run.side)
    run.main.synchronize()
    f = lambda name, n: run.export(name, torch.bfloat16, (2, n, 128))  # noqa: E731
    keys = torch.cat([f("k_outlier", 32), f("k_cache", 464), f("k_local", 17)], 1)
    vals = torch.cat([f("v_outlier", 32), f("v_cache", 464), f("v_local", 17)], 1)
    assert torch.equal(keys[:, 512], kr[0])
    # the same rows as one paged cache: 513 rows in 33 pages
    pool = torch.zeros((2, 33, 2, 16, 128), dtype=torch.bfloat16, device="cuda")
    for x, rows in zip(pool, (keys, vals)):
        full = torch.zeros((2, 528, 128), dtype=torch.bfloat16, device="cuda")
        full[:, :513] = rows
        x.copy_(full.view(2, 33, 16, 128).permute(1, 0, 2, 3))
    table = torch.arange(33, dtype=torch.int32, device="cuda")[None]
    dense = skv.paged_attention(qr, pool[0], pool[1], table, torch.tensor([513], dtype=torch.int32, device="cuda"),
                                torch.empty_like(qr))
    for h in range(2):
        s = slice(4 * h, 4 * h + 4)
        check_attention("bf16", f64(qr[0, s]), f64(dense[0, s]), None, f64(keys[h]), f64(vals[h]), 128 ** -0.5)
    # both round their probabilities or outputs to bf16: within two of the output bar of the layer's own tests
    assert (out.float() - dense.float()).abs().max() <= 2e-2
    run.layer.close()
