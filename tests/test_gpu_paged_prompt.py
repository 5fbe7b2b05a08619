"""Attention of many new tokens per sequence over a paged cache, on the GPU against its float64 form.

Tolerances, derived from the arithmetic: a score is an fp32 sum of d exact products, off by delta = scale d 2^-24
sum|q_i k_i| at most, and a probability by 2 delta of itself.  Probabilities are rounded to bf16 (2^-8); exp2 with exponents
below 2^6 and the fp32 sums of probabilities add less than 2^-16.  Sums of values are cut off after every 16 rows, 2^-22 of
what is there: n / 16 2^-22 for n rows.  So |out - ref| <= (2 delta + 2^-8 + 2^-16 + n 2^-26) sum p|v| + 2^-8 |ref|, and
lse within delta + 2^-16 + 2^-22 |lse|.
"""
import math

import numpy as np
import pytest
import torch

import sparse_kv_cache_gb300 as skv
from tests.paged_harness import Paged, f64

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def sight(n, tokens, window, sink):
    """[tokens][n]: which rows the last tokens of n rows see."""
    r, j = np.arange(n - tokens, n)[:, None], np.arange(n)[None]
    return (j <= r) & ((window == 0) | (j > r - window) | (j < sink))


def check(q, got, lse, k, v, seen, scale):
    """q [tokens][d] of one head over rows k, v [n][d]; got [tokens][d], lse [tokens]; seen [tokens][n]."""
    n, d = k.shape
    some = seen.any(1)
    assert (got[~some] == 0).all() and np.all(lse[~some] == -np.inf)
    q, got, lse, seen = q[some], got[some], lse[some], seen[some]
    if not len(q):
        return
    live = seen.any(0)
    k, v, seen = k[live], v[live], seen[:, live]
    z = np.where(seen, scale * (q @ k.T), -np.inf)
    top = z.max(1, keepdims=True)
    p = np.exp(z - top)
    total = p.sum(1, keepdims=True)
    p /= total
    out, want = p @ v, (top + np.log(total))[:, 0]
    delta = (d * 2.0 ** -24 * abs(scale) * np.where(seen, np.abs(q) @ np.abs(k).T, 0.0)).max(1)
    tol = (2 * delta[:, None] + 2.0 ** -8 + 2.0 ** -16 + n * 2.0 ** -26) * (p @ np.abs(v)) + 2.0 ** -8 * np.abs(out)
    assert not np.isnan(got).any()
    assert (np.abs(got - out) <= tol).all(), f"off by {np.abs(got - out).max():.3g}, {(np.abs(got - out) / tol).max():.3g} of the allowed"
    assert (np.abs(lse - want) <= delta + 2.0 ** -16 + 2.0 ** -22 * np.abs(want)).all()


def check_all(c, tokens, q, out, lse, window=0, sink=0, scale=None, heads=None):
    scale = scale or 1 / math.sqrt(c.d)
    start, G = np.concatenate([[0], np.cumsum(tokens)]), q.shape[1] // c.heads
    qf, of, lf = f64(q), f64(out), f64(lse)
    for b, n in enumerate(c.n):
        at = slice(start[b], start[b + 1])
        for h in range(c.heads):
            k, v = f64(c.krows[b][h]), f64(c.vrows[b][h])
            for g in range(h * G, (h + 1) * G) if heads is None else [h * G + heads % G]:
                check(qf[at, g], of[at, g], lf[at, g], k, v, sight(n, tokens[b], window, sink), scale)


def ask(c, G, tokens, seed=1, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((sum(tokens), c.heads * G, c.d), generator=g) * size).to(torch.bfloat16).cuda()


def attend(c, q, tokens, table=None, **kw):
    out, lse = torch.full_like(q, math.nan), torch.full(q.shape[:2], math.nan, device="cuda")
    start = i32(np.concatenate([[0], np.cumsum(tokens)]))
    skv.paged_prompt_attention(q, c.k, c.v, c.table if table is None else table, c.lens, start, out, lse, **kw)
    return out, lse


CASES = [
    # G, heads, d, ps, layout, lens, tokens, window, sink
    (4, 2, 128, 16, "hnd", [1], [1], 0, 0),
    (4, 2, 128, 16, "hnd", [5, 130, 0, 128], [5, 2, 0, 1], 0, 0),
    (1, 1, 64, 8, "nhd", [8, 9, 127, 128, 129, 1], [8, 3, 127, 1, 129, 1], 0, 0),
    (8, 1, 128, 8, "hnd", [300, 31, 0, 65], [300, 16, 0, 17], 0, 0),
    (3, 2, 64, 32, "nhd", [500, 43, 42, 85, 86], [100, 43, 42, 85, 86], 0, 0),
    (7, 1, 128, 64, "hnd", [1000, 37], [37, 36], 0, 0),
    (5, 1, 64, 128, "nhd", [700, 50], [51, 50], 0, 0),
    (6, 2, 128, 256, "hnd", [900, 600], [44, 22], 0, 0),
    (2, 1, 128, 1024, "hnd", [3000, 1500], [200, 129], 0, 0),
    (1, 8, 128, 16, "hnd", [1500, 257, 256, 255], [1500, 257, 256, 255], 0, 0),       # more units than SMs are free to split
    (4, 1, 128, 16, "hnd", [9000], [3], 0, 0),                                        # few rows, a long cache: parts
    (2, 2, 64, 8, "nhd", [4000, 3, 2000], [2, 1, 65], 0, 0),
    (4, 2, 128, 16, "hnd", [700, 130, 5], [700, 100, 5], 1, 0),
    (4, 2, 128, 16, "nhd", [700, 130, 5], [300, 100, 5], 64, 4),
    (2, 1, 64, 8, "hnd", [900, 300], [900, 130], 128, 130),
    (1, 2, 128, 64, "hnd", [1400, 600], [1100, 1], 333, 1),
    (8, 1, 64, 32, "nhd", [6000, 1200], [70, 33], 1000, 300),
    (4, 1, 128, 128, "hnd", [5000], [4], 3000, 5),                                    # parts of a window
    (4, 1, 128, 16, "hnd", [300, 20], [300, 20], 1 << 30, 7),
    (4, 1, 128, 16, "hnd", [300, 20], [300, 20], 5, (1 << 31) - 1),
    (2, 1, 64, 16, "hnd", [(i * 37) % 90 for i in range(300)], [min((i * 37) % 90, (i * 13) % 7) for i in range(300)], 0, 0),
    (4, 1, 128, 16, "hnd", [(i * i * 211) % 3001 for i in range(60)], [min((i * i * 211) % 3001, (i * 13) % 7) for i in range(60)], 0, 0),   # parts of uneven units
    (2, 2, 64, 32, "hnd", [20000, 0, 7, 129, 5000] + [i for i in range(20)], [5, 0, 7, 129, 66] + [i % 3 if i > 2 else 0 for i in range(20)], 0, 0),
    (4, 1, 128, 64, "nhd", [9000, 300, 4000, 20, 2500], [40, 33, 3, 20, 31], 2000, 600),
]


@pytest.mark.parametrize("G,heads,d,ps,layout,lens,tokens,window,sink", CASES)
def test_prompts_match_float64(G, heads, d, ps, layout, lens, tokens, window, sink):
    c = Paged("bf16", lens, heads, d, ps, layout, seed=len(lens) + G)
    q = ask(c, G, tokens)
    # what no token sees is NaN, and pages without a row that is seen are gone
    for b, n in enumerate(lens):
        live = sight(n, tokens[b], window, sink).any(0) if tokens[b] else np.zeros(n, bool)
        hidden = np.flatnonzero(~live)
        for pool in (c.k, c.v):
            if len(hidden):
                pool[c.table[b, torch.as_tensor(hidden // ps).cuda()].long(), :, torch.as_tensor(hidden % ps).cuda()] = math.nan
        gone = np.setdiff1d(np.arange(-(-n // ps)), np.flatnonzero(live) // ps)
        if len(gone):
            c.table[b, torch.as_tensor(gone).cuda()] = -1
    out, lse = attend(c, q, tokens, window=window, sink=sink)
    check_all(c, tokens, q, out, lse, window, sink)
    # a table with room for far longer sequences may be split another way
    wide = torch.cat([c.table, torch.full((len(lens), 65536 // ps), -1, dtype=torch.int32, device="cuda")], 1)
    out, lse = attend(c, q, tokens, wide, window=window, sink=sink)
    check_all(c, tokens, q, out, lse, window, sink)
    assert skv.paged_status() == 0


def test_a_long_prompt():
    c = Paged("bf16", [10000], 1, 128, 16, seed=3)
    q = ask(c, 4, [10000])
    for window, sink in ((0, 0), (2000, 4)):
        out, lse = attend(c, q, [10000], window=window, sink=sink)
        check_all(c, [10000], q, out, lse, window, sink, heads=2)


@pytest.mark.parametrize("scale,size", [(1.0, 1.0), (-0.3, 1.0), (0.088, 60.0), (1e-6, 1.0), (-1e-30, 1e30), (1e-30, 1e30)])
@pytest.mark.parametrize("window", [0, 50])
def test_scales_and_peaked_scores(scale, size, window):
    c = Paged("bf16", [513, 200], 2, 128, 16, seed=3)
    q = ask(c, 4, [300, 200], 5, size)
    out, lse = attend(c, q, [300, 200], scale=scale, window=window, sink=3)
    check_all(c, [300, 200], q, out, lse, window, 3, scale)


def test_scores_that_climb():
    c = Paged("bf16", [1500], 1, 128, 16, seed=4)
    c.krows[0][0] = torch.linspace(0.01, 6.0, 1500)[:, None].to(torch.bfloat16)
    for p in range(-(-1500 // 16)):
        rows = c.krows[0][0, 16 * p:16 * (p + 1)]
        c.k[int(c.table[0, p]), 0, :len(rows)] = rows.cuda()
    q = torch.ones((700, 2, 128), dtype=torch.bfloat16, device="cuda")
    for scale in (0.05, -0.05):
        out, lse = attend(c, q, [700], scale=scale)
        check_all(c, [700], q, out, lse, scale=scale)


def test_values_near_the_largest_do_not_overflow():
    c = Paged("bf16", [2000, 300], 1, 64, 16, seed=6)
    most = torch.finfo(torch.bfloat16).max
    c.v.copy_(torch.where(c.v.isnan(), c.v, most))
    c.vrows = [torch.full_like(x, most) for x in c.vrows]
    for tokens in ([500, 300], [1, 2]):
        q = ask(c, 4, tokens)
        out, lse = attend(c, q, tokens)
        assert out.isfinite().all()
        check_all(c, tokens, q, out, lse)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tokens", [3, 200, 700])
@pytest.mark.parametrize("window,sink", [(0, 0), (40, 3), (300, 130)])
def test_what_is_not_finite_reaches_those_who_see_it_alone(d, tokens, window, sink):
    """Infinities and NaN in values, scattered over the tiles: each changes its own dimension of the tokens that see its
    row, and nothing else."""
    n, G = 700, 2
    c = Paged("bf16", [n], 1, d, 16, seed=tokens + d)
    q = ask(c, G, [tokens], 7, 0.3)
    clean = c.vrows[0].clone()
    bad = [(699, 3, math.inf), (600, 5, -math.inf), (520, 6, math.nan), (1, 9, math.inf), (2, 9, -math.inf), (128, 11, math.inf),
           (511, d - 1, math.inf), (640, 0, math.nan)]
    for row, dim, x in bad:
        c.v[int(c.table[0, row // 16]), 0, row % 16, dim] = x
        clean[0, row, dim] = 0.0
    out, lse = attend(c, q, [tokens], window=window, sink=sink)
    seen = sight(n, tokens, window, sink)
    of, lf, qf = f64(out), f64(lse), f64(q)
    spoilt = np.zeros((tokens, d), bool)
    for dim in {x[1] for x in bad}:
        parts = [(row, x) for row, k, x in bad if k == dim]
        hit = seen[:, [row for row, _ in parts]]
        sums = np.where(hit, [x for _, x in parts], 0.0)
        with np.errstate(invalid="ignore"):
            want = sums.sum(1)
        spoilt[:, dim] = hit.any(1)
        for g in range(G):
            rows = hit.any(1)
            assert np.array_equal(of[rows, g, dim], want[rows], equal_nan=True)
    assert np.isfinite(of[~np.repeat(spoilt[:, None], G, 1)]).all()
    for g in range(G):
        k, v = f64(c.krows[0][0]), f64(clean[0])
        got = np.where(spoilt, 0.0, of[:, g])
        z = np.where(seen, (qf[:, g] @ k.T) / math.sqrt(d), -np.inf)
        p = np.exp(z - z.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        want = np.where(spoilt, 0.0, p @ v)
        # the values set to zero here are infinite there: only dimensions that saw none of them compare
        assert (np.abs(got - want) <= (2.0 ** -7 + 2.0 ** -11) * (p @ np.abs(v)) + 2.0 ** -8 * np.abs(want))[~spoilt].all()
    assert np.isfinite(lf).all() and skv.paged_status() == 0


def test_keys_that_are_not_finite():
    c = Paged("bf16", [300, 300, 300], 1, 64, 16, seed=7)
    q = ask(c, 2, [300, 300, 300], 8).abs() + 0.5
    c.k[int(c.table[0, 12]), 0, 8] = math.nan            # row 200: NaN for the tokens from it on
    c.k[int(c.table[1, 2]), 0, 1] = -math.inf            # row 33 weighs nothing
    out, lse = attend(c, q, [300, 300, 300])
    assert out[200:300].isnan().all() and lse[200:300].isnan().all() and not out[:200].isnan().any()
    live = np.arange(300) != 33
    seen = sight(300, 300, 0, 0)
    for g in range(2):
        check(f64(q[300:600, g]), f64(out[300:600, g]), f64(lse[300:600, g]), f64(c.krows[1][0])[live], f64(c.vrows[1][0])[live],
              seen[:, live], 0.125)
    c.k[:] = -math.inf
    out, lse = attend(c, q, [300, 300, 300])
    assert (out == 0).all() and (lse == -math.inf).all()


def test_bad_pages_and_starts_are_reported_and_not_followed():
    c = Paged("bf16", [300, 40], 1, 64, 16, seed=15)
    q = ask(c, 2, [100, 40])
    c.table[0, 1], c.table[0, 15] = -5, c.k.shape[0]
    live = np.r_[0:16, 32:240, 256:300]
    out, lse = attend(c, q, [100, 40])
    seen = sight(300, 100, 0, 0)[:, live]
    for g in range(2):
        check(f64(q[:100, g]), f64(out[:100, g]), f64(lse[:100, g]), f64(c.krows[0][0])[live], f64(c.vrows[0][0])[live], seen, 0.125)
        check(f64(q[100:, g]), f64(out[100:, g]), f64(lse[100:, g]), f64(c.krows[1][0]), f64(c.vrows[1][0]), sight(40, 40, 0, 0), 0.125)
    assert skv.paged_status() == -5 and skv.paged_status() == 0
    out = torch.full_like(q, 7.0)
    for start in ([0, 150, 160], [-3, 50, 60], [40, 0, 10]):
        skv.paged_prompt_attention(q, c.k, c.v, c.table[:, :1].contiguous(), i32([16, 16]), i32(start), out)
        assert skv.paged_status() == -5
    lens = i32([-1, 1000])
    skv.paged_prompt_attention(q, c.k, c.v, c.table, lens, i32([0, 1, 2]), out)
    assert skv.paged_status() == -5 and (out[0] == 0).all()


def test_more_tokens_than_rows_and_tokens_of_no_sequence():
    c = Paged("bf16", [10, 300], 2, 64, 16, seed=16)
    q = torch.randn((200, 4, 64), device="cuda").to(torch.bfloat16)
    out, lse = torch.full_like(q, 7.0), torch.full((200, 4), 7.0, device="cuda")
    skv.paged_prompt_attention(q, c.k, c.v, c.table, c.lens, i32([3, 103, 180]), out, lse)
    assert (out[:3] == 7).all() and (out[180:] == 7).all() and (lse[180:] == 7).all()
    assert (out[3:93] == 0).all() and (lse[3:93] == -math.inf).all()
    for h in range(2):
        for g in (2 * h, 2 * h + 1):
            check(f64(q[93:103, g]), f64(out[93:103, g]), f64(lse[93:103, g]), f64(c.krows[0][h]), f64(c.vrows[0][h]), sight(10, 10, 0, 0), 0.125)
            check(f64(q[103:180, g]), f64(out[103:180, g]), f64(lse[103:180, g]), f64(c.krows[1][h]), f64(c.vrows[1][h]), sight(300, 77, 0, 0), 0.125)
    assert skv.paged_status() == 0


def test_strided_queries_and_results():
    c = Paged("bf16", [333, 20], 2, 128, 16, "nhd", seed=10)
    fused = torch.randn((120, 16, 128), device="cuda").to(torch.bfloat16)
    q = fused[:, 4:12]                                     # a slice of a fused projection
    wide = torch.full((120, 8, 160), math.nan, dtype=torch.bfloat16, device="cuda")
    out, lse = wide[..., 16:144], torch.empty((120, 8), device="cuda")
    skv.paged_prompt_attention(q, c.k, c.v, c.table, c.lens, i32([0, 100, 120]), out, lse)
    check_all(c, [100, 20], q, out, lse)
    assert wide[..., :16].isnan().all() and wide[..., 144:].isnan().all()
    # one head, one token: strides that are never stepped through
    c = Paged("bf16", [30], 1, 64, 16, seed=44)
    odd = lambda t: t.as_strided(t.shape, (t.stride(0), 129, t.stride(2), 1))  # noqa: E731
    q = torch.randn((1, 1, 64), device="cuda").to(torch.bfloat16).as_strided((1, 1, 64), (77, 33, 1))
    out, lse = torch.empty_like(q), torch.empty((1, 1), device="cuda")
    skv.paged_prompt_attention(q, odd(c.k), odd(c.v), c.table, c.lens, i32([0, 1]), out, lse)
    check_all(c, [1], q, out, lse)


def test_pools_beyond_32_bit_offsets():
    n, d, ps, step = 300, 128, 16, 1 << 25
    c = Paged("bf16", [n], 1, d, ps, seed=13)
    big = [torch.empty(step * 80, dtype=torch.bfloat16, device="cuda").as_strided((80, 1, ps, d), (step, ps * d, d, 1)) for _ in range(2)]
    ids = [79, 3, 78, 70, 65, 77, 68, 1, 2, 4, 5, 6, 7, 8, 9, 10, 11, 12, 66]
    for pool, small in zip(big, (c.k, c.v)):
        for p in range(19):
            pool[ids[p]] = small[c.table[0, p].long()]
    c.k, c.v = big
    q = ask(c, 4, [120])
    out, lse = attend(c, q, [120], i32([ids]))
    check_all(c, [120], q, out, lse)


def test_streams_threads_and_bits():
    """The same bits on every stream and from every thread, with parts that share no workspace."""
    import threading
    c = Paged("bf16", [5000, 500, 0, 3000], 2, 128, 16, seed=18)
    tokens = [[3, 200, 0, 1], [1, 1, 0, 7]]
    qs = [ask(c, 4, t, 19 + i) for i, t in enumerate(tokens)]
    want = [attend(c, q, t) for q, t in zip(qs, tokens)]
    torch.cuda.synchronize()
    got, failed = [[], []], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                got[i] = [attend(c, qs[i], tokens[i]) for _ in range(30)]
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
        assert len(got[i]) == 30 and all(torch.equal(o, want[i][0]) and torch.equal(s, want[i][1]) for o, s in got[i])
    # handed-in streams
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[attend(c, qs[j], tokens[j], stream=streams[j]) for _ in range(3)] for j in range(2)]
    torch.cuda.synchronize()
    torch.cuda.synchronize()
    assert len(outs[0]) == 3


def test_captured_calls_replay_with_new_lengths():
    c = Paged("bf16", [700, 300], 2, 128, 16, seed=21)
    q = ask(c, 4, [100, 60], 22)
    start = i32([0, 100, 160])
    outs, lses = [torch.empty_like(q) for _ in range(2)], [torch.empty(q.shape[:2], device="cuda") for _ in range(2)]
    graphs = []
    for out, lse in zip(outs, lses):                       # two graphs, replayed on two streams at once
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            skv.paged_prompt_attention(q, c.k, c.v, c.table, c.lens, start, out, lse)
        graphs.append(g)
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    whole = c.krows, c.vrows
    for lens, tokens in (([700, 300], [100, 60]), ([1, 0], [1, 0]), ([333, 200], [5, 155]), ([100, 300], [60, 0])):
        c.lens.copy_(i32(lens))
        start.copy_(i32(np.concatenate([[0], np.cumsum(tokens)])))
        torch.cuda.synchronize()
        for g, st in zip(graphs, s):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        c.n = lens
        c.krows, c.vrows = ([x[:, :n] for x, n in zip(rows, lens)] for rows in whole)
        for out, lse in zip(outs, lses):
            check_all(c, tokens, q, out, lse)
    assert skv.paged_status() == 0


def test_a_prompt_and_its_steps_are_one_causal_attention():
    """Norm, rotation and append of a prompt in two chunks, its attention, then single steps and a draft of three tokens: all of
    them rows of one causal attention, through a window too."""
    H, G, d, n = 2, 4, 128, 400
    g = torch.Generator().manual_seed(2)
    make = lambda *s: torch.randn(s, generator=g).bfloat16().cuda()  # noqa: E731
    q, k, v, w = make(n, H * G, d), make(n, H, d), make(n, H, d), make(d)
    pools = [torch.full((30, H, 16, d), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table = torch.randperm(30, generator=g)[:25].to(torch.int32)[None].cuda()
    pos, q2 = torch.arange(n, dtype=torch.int32, device="cuda"), torch.empty_like(q)
    for window in (0, 90):
        outs, lses = [], []
        for lo, hi in ((0, 230), (230, 395), (395, 396), (396, 399), (399, 400)):
            at = slice(lo, hi)
            skv.qk_norm_rope(q[at], k[at], pos[at], q2[at], q_weight=w, k_weight=w, v=v[at], k_cache=pools[0], v_cache=pools[1],
                             table=table, seq=torch.zeros_like(pos[at]), index=pos[at])
            out, lse = torch.empty_like(q2[at]), torch.empty((hi - lo, H * G), device="cuda")
            if hi - lo > 1:
                skv.paged_prompt_attention(q2[at], *pools, table, i32([hi]), i32([0, hi - lo]), out, lse, window=window, sink=2)
            else:
                skv.paged_attention(q2[at], *pools, table, i32([hi]), out, lse, window=window, sink=2)
            outs.append(out)
            lses.append(lse)
        out, lse = torch.cat(outs), torch.cat(lses)
        rows = torch.arange(n, device="cuda")
        kr, vr = (pool[table[0, rows // 16].long(), :, rows % 16] for pool in pools)
        for h in range(H):
            for i in range(h * G, (h + 1) * G):
                check(f64(q2[:, i]), f64(out[:, i]), f64(lse[:, i]), f64(kr[:, h]), f64(vr[:, h]), sight(n, n, window, 2), d ** -0.5)
    assert skv.paged_status() == 0


def test_a_chunk_over_a_cache_of_codes():
    """A context kept in 8 bits is read back into pages, and a chunk of new tokens attends over it."""
    H, G, d, ps, n, new = 2, 4, 64, 16, 200, 56
    g = torch.Generator().manual_seed(5)
    make = lambda *s: torch.randn(s, generator=g).bfloat16().cuda()  # noqa: E731
    k, v, q = make(n, H, d), make(n, H, d), make(new, H * G, d)
    pools = [torch.zeros((16, H, ps, d), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.zeros((16, H, 2), device="cuda") for _ in range(2)]
    table = torch.randperm(16, generator=g)[:13].to(torch.int32)[None].cuda()
    skv.paged_quantise(k, v, *pools, *scales, table, i32([0]), i32([0, n]))
    back = [torch.zeros((13 * ps, H, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    skv.paged_dequantise(*pools, *scales, table, i32([n]), i32([0]), i32([0, 13 * ps]), *back)
    pages = [x.view(13, ps, H, d).transpose(1, 2) for x in back]              # token-major pages, in order
    out, lse = torch.empty_like(q), torch.empty((new, H * G), device="cuda")
    skv.paged_prompt_attention(q, *pages, i32([range(13)]), i32([n]), i32([0, new]), out, lse)
    for h in range(H):
        for i in range(h * G, (h + 1) * G):
            check(f64(q[:, i]), f64(out[:, i]), f64(lse[:, i]), f64(back[0][:n, h]), f64(back[1][:n, h]), sight(n, new, 0, 0), d ** -0.5)
    assert skv.paged_status() == 0


def test_other_types_and_host_memory_are_refused():
    for kind in ("f32", "fp8"):
        c = Paged(kind, [20], 1, 64, 16, seed=1)
        q = torch.zeros((2, 2, 64), dtype=c.k.dtype, device="cuda")
        with pytest.raises(skv.ShadowKVError) as e:
            attend(c, q, [2])
        assert e.value.code == -8
    c = Paged("bf16", [20], 1, 64, 16, seed=1)
    q, start = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda"), i32([0, 2])
    args = dict(q=q, k_cache=c.k, v_cache=c.v, table=c.table, lens=c.lens, start=start, out=torch.empty_like(q))
    for bad in (dict(q=q.cpu()), dict(k_cache=c.k.cpu()), dict(table=c.table.cpu()), dict(lens=c.lens.cpu()), dict(start=start.cpu()),
                dict(out=q.cpu())):
        with pytest.raises(skv.ShadowKVError) as e:
            skv.paged_prompt_attention(**{**args, **bad})
        assert e.value.code == -1
