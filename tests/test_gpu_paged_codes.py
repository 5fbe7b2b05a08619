"""Paged caches of 8-bit codes -- written, read back, attended over -- and attention over a window and first rows, on
the GPU against float64 forms.

Tolerances, derived from the arithmetic:

* writing: scales are powers of two, so x / scale is exact and a code is x rounded once: codes and scales are equal.
* reading back: code * scale is exact in fp32 (4 bits and a power of two); bf16 holds 4 bits: equal.
* attention over codes: as in test_gpu_paged.py, delta = scale d 2^-24 sum|q_i k_i| for the fp32 sum of a score (its
  products are exact), and besides 2^-22 of a score for its two factors (scale of the block, power of two of
  the query, both exact powers of two here, but the products with them may round), and what fp16 loses of
  queries 2^-39 below their head's largest: scale d 2^-39 max|q| max|k|.  Probabilities times scales are rounded to fp16:
  2^-11 of each, or 2^-25 against a top of 2^7 at least, so 2^-32 of the largest on each code.  Exponents up to 128
  have roundings of 2^-17, with exp2 and the fp32 sums below 2^-15.  One rounding to bf16: 2^-8 of the result.
* windows: the tolerances of test_gpu_paged.py over the rows that are seen.
"""
import math

import numpy as np
import pytest
import torch

import sparse_kv_cache_gb300 as skv
from oracle import paged_ref as ref
from tests.paged_harness import Paged, f64
from tests.test_gpu_paged import check_attention, queries

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Codes:
    """A paged cache of random codes and scales.  Codes that no row uses are NaN, and so are scales of blocks without
    a row; table entries without a page are -1."""

    def __init__(self, lens, heads, d, ps, block, layout="hnd", seed=0, cap=0, spread=3):
        g = torch.Generator().manual_seed(seed)
        self.n, self.heads, self.d, self.ps, self.block = list(lens), heads, d, ps, block
        own = [-(-max(n, cap) // ps) for n in self.n]
        pages = sum(own) + 2
        ids = torch.randperm(pages, generator=g).to(torch.int32)
        table = torch.full((len(self.n), max(1, *own)), -1, dtype=torch.int32)
        at = 0
        for b, k in enumerate(own):
            table[b, :k] = ids[at:at + k]
            at += k
        nb = ps // block
        self.codes, self.scales = {}, {}
        pools = {}
        for name in "kv":
            pool = torch.full((pages, heads, ps, d), 0x7F, dtype=torch.uint8)
            scale = torch.full((pages, heads, nb), math.nan)
            self.codes[name], self.scales[name] = [], []
            for b, n in enumerate(self.n):
                x = (torch.randn((heads, n, d), generator=g) * 100).clamp(-448, 448).to(E4M3)
                s = torch.exp2(torch.randint(-6 - spread, -5 + spread, (heads, -(-n // block)), generator=g).float())
                self.codes[name].append(x)
                self.scales[name].append(s)
                for p in range(-(-n // ps)):
                    lo, hi = p * ps, min(n, (p + 1) * ps)
                    pool[table[b, p], :, :hi - lo] = x[:, lo:hi].view(torch.uint8)
                    part = s[:, lo // block:-(-hi // block)]
                    scale[table[b, p], :, :part.shape[1]] = part
            if layout == "nhd":
                pool = pool.transpose(1, 2).contiguous().transpose(1, 2)
            pools[name] = pool.cuda().view(E4M3), scale.cuda()
        (self.k, self.ks), (self.v, self.vs) = pools["k"], pools["v"]
        self.table, self.lens = table.cuda(), i32(self.n)
        self.cache = dict(k_cache=self.k, v_cache=self.v, k_scale=self.ks, v_scale=self.vs, table=self.table, lens=self.lens)

    def rows(self, name, b, h):
        """(codes, scale of each row) of a unit, float64."""
        x = self.codes[name][b][h].float().double().numpy()
        return x, self.scales[name][b][h].double().numpy().repeat(self.block)[:len(x)]

    def held(self, name, b, h, n):
        """The first n rows of a unit, and their scales, as they are stored now."""
        pool, scale = (self.k, self.ks) if name == "k" else (self.v, self.vs)
        at = torch.arange(n)
        page = self.table.cpu()[b, at // self.ps].long()
        codes = pool.view(torch.uint8).cpu()[page, h, at % self.ps].view(E4M3).float().double().numpy()
        return codes, scale.cpu()[page, h, at % self.ps // self.block].double().numpy()


def check_unit(q, got, lse, k, ks, v, vs, scale):
    """q [G][d] over rows of codes k, v with scales ks, vs; got [G][d], lse [G]."""
    out, want, p = ref.attend(q, k * ks[:, None], v * vs[:, None], scale)
    if len(k) == 0:
        assert (got == 0).all() and np.all(lse == -np.inf)
        return
    d = q.shape[1]
    size = np.abs(q) @ np.abs(k * ks[:, None]).T
    delta = abs(scale) * (d * 2.0 ** -24 + 2.0 ** -22) * size.max(1) + \
        abs(scale) * d * 2.0 ** -39 * np.abs(q).max(1) * np.abs(k * ks[:, None]).max()
    lost = 2.0 ** -32 * (p * vs).max(1)[:, None] * np.abs(v).sum(0)[None]
    tol = (2 * delta[:, None] + 2.0 ** -11 + 2.0 ** -15) * (p @ np.abs(v * vs[:, None])) + 2.0 ** -8 * np.abs(out) + lost
    assert not np.isnan(got).any()
    assert (np.abs(got - out) <= tol).all(), f"off by {np.abs(got - out).max():.3g}, {(np.abs(got - out) / tol).max():.3g} of the allowed"
    assert (np.abs(lse - want) <= delta + 2.0 ** -16 + 2.0 ** -22 * np.abs(want)).all()


def check_codes(c, q, out, lse, scale=None, window=0, sink=0):
    G, scale = q.shape[1] // c.heads, scale or 1 / math.sqrt(c.d)
    qf, of, lf = f64(q), f64(out), f64(lse)
    for b, n in enumerate(c.n):
        live = ref.seen_rows(n - 1, window, sink)
        for h in range(c.heads):
            s = slice(h * G, (h + 1) * G)
            (k, ks), (v, vs) = c.rows("k", b, h), c.rows("v", b, h)
            check_unit(qf[b, s], of[b, s], lf[b, s], k[live], ks[live], v[live], vs[live], scale)


def ask(c, G, seed=1, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((len(c.n), c.heads * G, c.d), generator=g) * size).to(torch.bfloat16).cuda()


def attend(c, q, **kw):
    out, lse = torch.full_like(q, math.nan), torch.full(q.shape[:2], math.nan, device="cuda")
    skv.paged_attention(q, out=out, lse=lse, **c.cache, **kw)
    return out, lse


# ------------------------------------------------------------------ attention over codes

CASES = [
    (4, 2, 128, 16, 16, "hnd", [1]),
    (1, 1, 64, 8, 8, "nhd", [8, 9, 15, 16, 17, 1]),
    (8, 2, 128, 8, 8, "hnd", [63, 64, 65, 0, 127, 128, 129]),
    (3, 3, 128, 32, 8, "nhd", [1000, 0, 0, 5, 333]),
    (7, 1, 64, 1024, 128, "hnd", [2049, 1023]),
    (8, 1, 128, 16, 8, "hnd", [8190]),
    (2, 2, 128, 64, 32, "nhd", [40000, 1, 0, 700]),
    (5, 8, 128, 16, 16, "hnd", [300] * 40 + [0] * 200),
    (4, 1, 64, 16, 16, "hnd", [0] * 150 + [77] + [0] * 150 + [3000]),
    (1, 1, 64, 8, 8, "hnd", [(i * 7919) % 41 for i in range(1000)]),
    (8, 4, 128, 128, 64, "hnd", [(i * 97) % 700 for i in range(150)]),
    (6, 2, 64, 256, 128, "nhd", [5000, 257]),
]


@pytest.mark.parametrize("G,heads,d,ps,block,layout,lens", CASES)
def test_attention_over_codes(G, heads, d, ps, block, layout, lens):
    c = Codes(lens, heads, d, ps, block, layout, seed=len(lens) + G)
    q = ask(c, G)
    check_codes(c, q, *attend(c, q))
    # a table with room for far longer sequences: the form without clusters
    c.cache["table"] = torch.cat([c.table, torch.full((len(lens), 16384 // ps), -1, dtype=torch.int32, device="cuda")], 1)
    check_codes(c, q, *attend(c, q))
    assert skv.paged_status() == 0


@pytest.mark.parametrize("scale,size,spread", [(1.0, 1.0, 3), (-0.3, 1.0, 3), (0.088, 60.0, 1), (1e-6, 1.0, 3), (0.05, 1e-6, 40),
                                               (1e-30, 1e30, 2)])
def test_codes_with_scales_peaked_scores_and_far_apart_blocks(scale, size, spread):
    c = Codes([513, 200], 2, 128, 16, 8, seed=3, spread=spread)
    q = ask(c, 4, 5, size)
    if spread > 10:                      # scores that stay in range: keys alike, values far apart
        c.ks.copy_(torch.where(c.ks.isnan(), c.ks, 2.0 ** -5))
        c.scales["k"] = [torch.full_like(s, 2.0 ** -5) for s in c.scales["k"]]
    check_codes(c, q, *attend(c, q, scale=scale), scale)


def test_the_heaviest_scale_may_have_the_smallest_probability():
    """Rows of probability 2^-60 whose values, 2^70 times larger, carry the result; both orders."""
    for flip in (False, True):
        c = Codes([64], 1, 64, 16, 8, seed=5)
        k, ks, vs = torch.zeros((1, 64, 64)), torch.ones((1, 8)), torch.ones((1, 8))
        late = slice(0, 32) if flip else slice(32, 64)
        k[0, :, 0] = 60.0
        k[0, late, 0] = 0.0
        vs[0, 0 if flip else 4] = 2.0 ** 70
        c.codes["k"], c.scales["k"], c.scales["v"] = [k.to(E4M3)], [ks], [vs]
        for p in range(4):
            c.k.view(torch.uint8)[c.table[0, p], 0] = k.to(E4M3).view(torch.uint8)[0, 16 * p:16 * p + 16].cuda()
            c.ks[c.table[0, p], 0] = ks[0, 2 * p:2 * p + 2].cuda()
            c.vs[c.table[0, p], 0] = vs[0, 2 * p:2 * p + 2].cuda()
        q = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device="cuda")
        q[..., 0] = 1.0
        out, lse = attend(c, q, scale=math.log(2.0))
        check_codes(c, q, out, lse, math.log(2.0))
        assert f64(out).max() > 100.0


def test_largest_codes_and_scales_do_not_overflow():
    c = Codes([3000], 1, 64, 16, 16, seed=6)
    c.vs.copy_(torch.where(c.vs.isnan(), c.vs, 2.0 ** 119))      # 448 * 2^119 is below bf16's largest
    c.scales["v"] = [torch.full_like(s, 2.0 ** 119) for s in c.scales["v"]]
    c.v.view(torch.uint8)[:] = 0x7E
    c.codes["v"] = [torch.full_like(x.float(), 448.0).to(E4M3) for x in c.codes["v"]]
    q = ask(c, 4)
    for table in (c.table, torch.cat([c.table, c.table.new_full((1, 4096), -1)], 1)):
        c.cache["table"] = table
        out, lse = attend(c, q)
        check_codes(c, q, out, lse)


def test_nan_codes_and_queries_propagate():
    c = Codes([100, 100, 100], 1, 64, 16, 16, seed=7)
    q = ask(c, 2).abs() + 0.5
    c.k.view(torch.uint8)[c.table[0, 1].item(), 0, 3] = 0x7F
    c.v.view(torch.uint8)[c.table[1, 1].item(), 0, 3, 5] = 0x7F
    q[2, 1, 9] = math.nan
    out, lse = attend(c, q)
    assert out[0].isnan().all() and lse[0].isnan().all()
    assert out[1, :, 5].isnan().all() and not out[1, :, :5].isnan().any() and not out[1, :, 6:].isnan().any()
    assert out[2, 1].isnan().all() and not out[2, 0].isnan().any()


def test_bad_pages_of_codes_are_left_out():
    c = Codes([64, 40], 1, 64, 16, 8, seed=15)
    q = ask(c, 2, 16)
    c.table[0, 1], c.table[0, 3] = -5, c.k.shape[0]
    live = np.r_[0:16, 32:48]
    out, lse = attend(c, q)
    (k, ks), (v, vs) = c.rows("k", 0, 0), c.rows("v", 0, 0)
    check_unit(f64(q[0]), f64(out[0]), f64(lse[0]), k[live], ks[live], v[live], vs[live], 0.125)
    assert skv.paged_status() == -5 and skv.paged_status() == 0


# ------------------------------------------------------------------ windows

@pytest.mark.parametrize("kind", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("G,heads,d,ps,layout,lens,window,sink", [
    (4, 2, 128, 16, "hnd", [1, 2, 0, 16, 17, 40], 1, 0),
    (1, 1, 64, 8, "nhd", [300, 8, 9, 25], 8, 1),
    (8, 1, 128, 8, "hnd", [1000, 31, 32, 33], 17, 20),
    (3, 2, 64, 64, "hnd", [5000, 100, 64, 0], 1000, 4),
    (4, 1, 128, 1024, "nhd", [9000, 3000, 4097], 4096, 4),
    (2, 2, 128, 16, "hnd", [(i * 97) % 700 for i in range(150)], 65, 130),
    (5, 4, 64, 32, "nhd", [4000] * 150, 250, 3),
    (4, 2, 128, 16, "hnd", [40000, 30000, 1, 0], 20000, 100),
    (4, 2, 128, 16, "hnd", [100, 20], 1 << 30, 7),
    (4, 2, 128, 16, "hnd", [100, 20], 5, (1 << 31) - 1),
])
def test_windows(kind, G, heads, d, ps, layout, lens, window, sink):
    c = Paged(kind, lens, heads, d, ps, layout, seed=len(lens) + G)
    q = queries(c, G)
    qf = f64(q)
    # nothing between the first and the last rows is read: NaN there, and pages without a row that is seen are gone
    for b, n in enumerate(lens):
        live = ref.seen_rows(n - 1, window, sink)
        hidden = np.setdiff1d(np.arange(n), live)
        for pool in (c.k, c.v):
            raw = pool.view(torch.uint8) if pool.dtype == torch.float8_e5m2 else pool
            if len(hidden):
                page = c.table[b, torch.as_tensor(hidden // ps).cuda()].long()
                raw[page, :, torch.as_tensor(hidden % ps).cuda()] = 0x7E if raw.dtype == torch.uint8 else math.nan
        gone = np.setdiff1d(np.arange(-(-n // ps)), live // ps)
        if len(gone):
            c.table[b, torch.as_tensor(gone).cuda()] = -1
    wide = torch.cat([c.table, torch.full((len(lens), 16384 // ps), -1, dtype=torch.int32, device="cuda")], 1)
    for table in (c.table, wide):
        out, lse = torch.full_like(q, math.nan), torch.full(q.shape[:2], math.nan, device="cuda")
        skv.paged_attention(q, c.k, c.v, table, c.lens, out, lse, window=window, sink=sink)
        of, lf = f64(out), f64(lse)
        for b, n in enumerate(lens):
            live = ref.seen_rows(n - 1, window, sink)
            for h in range(heads):
                s = slice(h * G, (h + 1) * G)
                check_attention(kind, qf[b, s], of[b, s], lf[b, s], f64(c.krows[b][h])[live], f64(c.vrows[b][h])[live], d ** -0.5)
    assert skv.paged_status() == 0


@pytest.mark.parametrize("G,heads,d,ps,block,layout,lens,window,sink", [
    (4, 2, 128, 16, 8, "hnd", [1, 2, 0, 16, 17, 40], 1, 0),
    (8, 1, 64, 8, 8, "nhd", [1000, 31, 32, 33], 17, 20),
    (3, 2, 128, 64, 64, "hnd", [5000, 100, 64, 0], 1000, 4),
    (2, 2, 128, 16, 16, "nhd", [(i * 97) % 700 for i in range(150)], 65, 130),
    (4, 2, 64, 32, 8, "hnd", [40000, 30000, 1, 0], 20000, 100),
])
def test_windows_over_codes(G, heads, d, ps, block, layout, lens, window, sink):
    c = Codes(lens, heads, d, ps, block, layout, seed=len(lens) + G)
    for b, n in enumerate(lens):
        live = ref.seen_rows(n - 1, window, sink)
        gone = np.setdiff1d(np.arange(-(-n // ps)), live // ps)
        if len(gone):
            c.table[b, torch.as_tensor(gone).cuda()] = -1
    q = ask(c, G)
    for more in (0, 16384 // ps):
        c.cache["table"] = torch.cat([c.table, torch.full((len(lens), more), -1, dtype=torch.int32, device="cuda")], 1)
        check_codes(c, q, *attend(c, q, window=window, sink=sink), None, window, sink)
    assert skv.paged_status() == 0


def test_a_window_over_everything_is_the_whole_cache():
    """The same rows in the same split: the same bits as without a window."""
    for kind in ("bf16", "fp8", "f32"):
        c = Paged(kind, [700, 64, 0, 9000], 2, 128, 16, seed=21)
        q = queries(c, 4, 22)
        whole = skv.paged_attention(q, c.k, c.v, c.table, c.lens, torch.empty_like(q))
        assert torch.equal(whole, skv.paged_attention(q, c.k, c.v, c.table, c.lens, torch.empty_like(q), window=9000))
        assert torch.equal(whole, skv.paged_attention(q, c.k, c.v, c.table, c.lens, torch.empty_like(q), window=1 << 30, sink=3))


# ------------------------------------------------------------------ writing and reading back

def quantised(c, b, h, name, start_row, new):
    """Codes and scales of a unit's rows after `new` [n][d] joined it at start_row."""
    codes, scales = c.rows(name, b, h)
    codes, scales = codes[:start_row], scales[:start_row]
    row, end = start_row, start_row + len(new)
    while row < end:
        lo = row // c.block * c.block
        hi = min(end, lo + c.block)
        got, size = ref.append_block(codes[lo:row], scales[lo] if row > lo else 0.0, new[row - start_row:hi - start_row])
        codes, scales = np.concatenate([codes[:lo], got]), np.concatenate([scales[:lo], np.full(hi - lo, size)])
        row = hi
    return codes, scales


WRITES = [
    ([0], [1], 2, 128, 16, 16, "hnd"),
    ([5, 0, 17, 8, 100], [1, 1, 1, 1, 1], 3, 64, 8, 8, "nhd"),
    ([0, 3, 0, 64, 31], [700, 0, 5, 64, 33], 2, 128, 32, 8, "hnd"),
    ([129, 1, 127], [300, 127, 1], 1, 128, 128, 128, "hnd"),
    ([1000, 0, 7], [25, 2049, 1500], 2, 64, 1024, 64, "nhd"),
    ([(i * 31) % 50 for i in range(700)], [(i * 7) % 4 for i in range(700)], 1, 64, 16, 16, "hnd"),
    ([40] * 40, [3] * 40, 2, 128, 64, 32, "nhd"),
]


@pytest.mark.parametrize("wide", ["bf16", "f32"])
@pytest.mark.parametrize("held,n,heads,d,ps,block,layout", WRITES)
def test_writing_and_reading_back(wide, held, n, heads, d, ps, block, layout):
    dt = torch.bfloat16 if wide == "bf16" else torch.float32
    cap = max(a + b for a, b in zip(held, n))
    c = Codes(held, heads, d, ps, block, layout, seed=sum(n) + block, cap=cap)
    start, T = np.concatenate([[0], np.cumsum(n)]), sum(n)
    g = torch.Generator().manual_seed(T + 1)
    # tokens of very different size, so that scales grow in the middle of blocks, and what has no code
    fused = torch.randn((T + 2, 2, heads + 1, d), generator=g) * torch.exp2(torch.randint(-12, 6, (T + 2, 2, heads + 1, 1), generator=g).float())
    fused[::5] *= 1e-3
    if T > 30:
        fused[7, 0, 0, 3], fused[8, 1, 0, 5], fused[9, 0, 0, 1] = math.inf, -math.inf, math.nan
        fused[11], fused[12] = 0.0, 1e-38
        fused[13, :, :, 0] = 2e38
    fused = fused.to(dt).cuda()
    k, v = fused[:T, 0, :heads], fused[:T, 1, 1:heads + 1]
    before = {name: (getattr(c, name).clone(), getattr(c, name + "s").clone()) for name in "kv"}
    skv.paged_quantise(k, v, c.k, c.v, c.ks, c.vs, c.table, c.lens, i32(start))
    assert skv.paged_status() == 0
    touched = {name: torch.zeros(c.k.shape[:3], dtype=torch.bool) for name in "kv"}
    table = c.table.cpu()
    first = [max(0, a - 3) for a in held]
    m = [a + x - f for a, x, f in zip(held, n, first)]
    back = [torch.full((sum(m) + 1, heads, d), 7.0, dtype=dt, device="cuda") for _ in range(2)]
    lens = i32([a + x for a, x in zip(held, n)])
    s2 = np.concatenate([[0], np.cumsum(m)])
    skv.paged_dequantise(c.k, c.v, c.ks, c.vs, c.table, lens, i32(first), i32(s2), *back)
    assert skv.paged_status() == 0
    for i, (name, x) in enumerate((("k", k), ("v", v))):
        xf, bf = f64(x), f64(back[i])
        for b in range(len(n)):
            rows = held[b] + n[b]
            for h in range(heads):
                want, size = quantised(c, b, h, name, held[b], xf[start[b]:start[b + 1], h])
                got, gs = c.held(name, b, h, rows)
                live = np.arange(rows) >= held[b] // block * block if n[b] else np.zeros(rows, bool)
                assert np.array_equal(got, want, equal_nan=True) and np.array_equal(gs, size)
                values = want * size[:, None]
                values = values if dt == torch.float32 else f64(torch.from_numpy(values).to(dt))
                assert np.array_equal(bf[s2[b]:s2[b + 1], h], values[first[b]:].astype(np.float32).astype(np.float64), equal_nan=True)
            at = torch.arange(rows)[live]
            touched[name][table[b, at // ps].long(), :, at % ps] = True
        assert (back[i][-1] == 7.0).all()
        # everything else is as it was
        pool, scale = before[name]
        same = getattr(c, name).view(torch.uint8).cpu() == pool.view(torch.uint8).cpu()
        assert same[~touched[name]].all()
        blocks = touched[name].unflatten(2, (-1, block)).any(-1)
        a, b_ = getattr(c, name + "s").cpu()[~blocks], scale.cpu()[~blocks]
        assert torch.equal(a.nan_to_num(-1.0), b_.nan_to_num(-1.0))


def test_a_row_at_a_time_is_the_same_block_in_the_end():
    """A block filled by single steps has the scale of its largest row, and codes that lose only what falls below the
    smallest code of the scales in between."""
    d, rows = 64, 37
    c = Codes([0], 2, d, 16, 16, seed=1, cap=rows)
    whole = Codes([0], 2, d, 16, 16, seed=1, cap=rows)
    g = torch.Generator().manual_seed(2)
    x = (torch.randn((rows, 2, d), generator=g) * torch.exp2(torch.randint(-2, 3, (rows, 2, 1), generator=g).float())).bfloat16().cuda()
    for t in range(rows):
        skv.paged_quantise(x[t:t + 1], x[t:t + 1], c.k, c.v, c.ks, c.vs, c.table, i32([t]), i32([0, 1]))
    skv.paged_quantise(x, x, whole.k, whole.v, whole.ks, whole.vs, whole.table, i32([0]), i32([0, rows]))
    for h in range(2):
        (a, sa), (b, sb) = c.held("k", 0, h, rows), whole.held("k", 0, h, rows)
        assert np.array_equal(sa, sb)
        # each rounding to subnormal codes is off by half a step of 2^-9, and there are few of them
        assert (np.abs(a - b) <= np.where(np.abs(b) >= 2.0 ** -5, 0.0, 4 * 2.0 ** -10)).all()


def test_what_is_out_of_range_is_not_written():
    c = Codes([10, 20], 1, 64, 16, 16, seed=4, cap=32)
    x = torch.ones((40, 1, 64), dtype=torch.bfloat16, device="cuda")
    start = i32([0, 4, 8])
    quiet = lambda: skv.paged_status() == 0  # noqa: E731
    def write(lens=(10, 20), start=start, table=None):  # noqa: E306
        pools = [c.k.clone(), c.v.clone(), c.ks.clone(), c.vs.clone()]
        skv.paged_quantise(x, x, *pools, c.table if table is None else table, i32(lens), start)
        return [(a.view(torch.uint8) if a.dtype == E4M3 else a.view(torch.int32)) !=
                (b.view(torch.uint8) if b.dtype == E4M3 else b.view(torch.int32)) for a, b in zip(pools, (c.k, c.v, c.ks, c.vs))]
    assert quiet()
    write()
    assert quiet()
    changed = write(lens=(30, 20))                       # two rows fit, two do not
    assert skv.paged_status() == -5
    assert changed[0][c.table[0, 1].long(), 0, 14:].all()
    for bad in ([0, 50, 60], [-3, 4, 8], [4, 0, 2]):     # tokens that there are not, and a start that falls
        write(start=i32(bad))
        assert skv.paged_status() == -5
    table = c.table.clone()
    table[0, 0], table[1, 1] = -1, c.k.shape[0]
    changed = write(table=table)
    assert skv.paged_status() == -5 and not changed[0].any() and not changed[2].any()
    write(lens=(-1, 33))
    assert skv.paged_status() == -5
    # reading back
    out = [torch.full((40, 1, 64), 7.0, device="cuda") for _ in range(2)]
    read = lambda lens, first, start, table=c.table: skv.paged_dequantise(  # noqa: E731
        c.k, c.v, c.ks, c.vs, table, i32(lens), i32(first), i32(start), *out)
    read([10, 20], [0, 0], [0, 12, 40])                  # more tokens than rows
    assert quiet() and (out[0][10:12] == 7.0).all() and (out[0][32:] == 7.0).all() and not (out[0][12:32] == 7.0).all()
    out[0].fill_(7.0)
    read([10, 20], [-1, 0], [0, 4, 8])
    assert skv.paged_status() == -5 and (out[0][:4] == 7.0).all() and not (out[0][4:8] == 7.0).all()
    out[0].fill_(7.0)
    read([10, 20], [0, 30], [0, 50, 60])
    assert skv.paged_status() == -5 and (out[0] == 7.0).all()
    read([10, 20], [0, 0], [0, 4, 8], table)
    assert skv.paged_status() == -5 and (out[0][:4] == 7.0).all() and not (out[0][4:8] == 7.0).all()


def test_tokens_of_no_sequence_are_left_out():
    """Tokens before start[0] and behind start[batch], more of them than the sequences have rows: places without a block,
    which look at no table."""
    for block, n in ((8, 300), (64, 1000)):
        c = Codes([5, 0, 33], 2, 64, 64, block, seed=block, cap=128)
        guard = torch.full((7, 2 + c.table.shape[1]), 1 << 29, dtype=torch.int32, device="cuda")    # bad ids around the table
        guard[2:5, 1:-1] = c.table
        table = guard[2:5, 1:-1]
        start = np.array([n, n + 4, n + 4, n + 24])
        x = torch.randn((n + 24 + 500, 2, 64), device="cuda").to(torch.bfloat16)
        before = c.k.clone()
        skv.paged_quantise(x, x, c.k, c.v, c.ks, c.vs, table, c.lens, i32(start))
        assert skv.paged_status() == 0
        back = [torch.full_like(x, 7.0) for _ in range(2)]
        skv.paged_dequantise(c.k, c.v, c.ks, c.vs, table, i32([9, 0, 53]), c.lens, i32(start), *back)
        assert skv.paged_status() == 0
        for b, held in ((0, 5), (2, 33)):
            for h in range(2):
                want, size = quantised(c, b, h, "k", held, f64(x[start[b]:start[b + 1], h]))
                got, gs = c.held("k", b, h, len(want))
                assert np.array_equal(got, want) and np.array_equal(gs, size)
                assert np.array_equal(f64(back[0][start[b]:start[b + 1], h]), (want * size[:, None])[held:])
        assert (back[0][:n] == 7.0).all() and (back[0][n + 24:] == 7.0).all()
        used = torch.zeros(c.k.shape[:3], dtype=torch.bool)
        for b, rows in ((0, 9), (2, 53)):
            at = torch.arange(rows)
            used[c.table.cpu()[b, at // 64].long(), :, at % 64] = True
        assert (c.k.view(torch.uint8).cpu() == before.view(torch.uint8).cpu())[~used].all()


def test_codes_beyond_32_bit_offsets():
    """Pages 2^26 bytes apart: their offsets pass 2^32."""
    n, d, ps, step = 100, 128, 16, 1 << 26
    c = Codes([n], 1, d, ps, 8, seed=13)
    big = [torch.empty(step * 80, dtype=torch.uint8, device="cuda").view(E4M3).as_strided((80, 1, ps, d), (step, ps * d, d, 1)) for _ in range(2)]
    scales = [torch.full((80, 1, 2), math.nan, device="cuda") for _ in range(2)]
    ids = [79, 3, 78, 70, 65, 77, 68]
    for big_, small, s_, t_ in zip(big, (c.k, c.v), scales, (c.ks, c.vs)):
        for p in range(7):
            big_.view(torch.uint8)[ids[p]] = small.view(torch.uint8)[c.table[0, p].long()]
            s_[ids[p]] = t_[c.table[0, p].long()]
    table = i32([ids])
    q = ask(c, 4, 14)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    go = lambda: skv.paged_attention(q, *big, table, c.lens, out, lse, k_scale=scales[0], v_scale=scales[1])  # noqa: E731
    go()
    check_codes(c, q, out, lse)
    x = torch.randn((12, 1, d), device="cuda").to(torch.bfloat16)
    skv.paged_quantise(x, x, *big, *scales, table, i32([n]), i32([0, 12]))
    back = [torch.empty_like(x) for _ in range(2)]
    skv.paged_dequantise(*big, *scales, table, i32([n + 12]), i32([n]), i32([0, 12]), *back)
    want, size = quantised(c, 0, 0, "k", n, f64(x[:, 0]))
    assert np.array_equal(f64(back[0][:, 0]), (want * size[:, None])[n:]) and skv.paged_status() == 0


# ------------------------------------------------------------------ as they are used

def test_prompts_then_steps_over_codes():
    """Prompts written, then steps: a row of each sequence written and attended over, whole and through a window,
    captured and replayed with new lengths and rows, on another stream."""
    B, H, G, d, ps, block, cap = 3, 2, 4, 128, 16, 16, 400
    lens = [300, 1, 47]
    c = Codes([0] * B, H, d, ps, block, seed=31, cap=cap)
    g = torch.Generator().manual_seed(8)
    make = lambda *s: torch.randn(s, generator=g).bfloat16().cuda()  # noqa: E731
    k, v = make(sum(lens), H, d), make(sum(lens), H, d)
    skv.paged_quantise(k, v, c.k, c.v, c.ks, c.vs, c.table, c.lens, i32(np.concatenate([[0], np.cumsum(lens)])))
    q, k1, v1 = torch.empty((B, H * G, d), dtype=torch.bfloat16, device="cuda"), make(B, H, d), make(B, H, d)
    rows, start = i32(lens), i32(range(B + 1))
    outs, lses = [torch.empty_like(q) for _ in range(2)], [torch.empty((B, H * G), device="cuda") for _ in range(2)]
    after = torch.empty_like(rows)

    def step():
        skv.paged_quantise(k1, v1, c.k, c.v, c.ks, c.vs, c.table, rows, start)
        torch.add(rows, 1, out=after)
        for out, lse, window in ((outs[0], lses[0], 0), (outs[1], lses[1], 33)):
            skv.paged_attention(q, c.k, c.v, c.table, after, out, lse, k_scale=c.ks, v_scale=c.vs, window=window, sink=4)
        rows.copy_(after)

    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in range(20):
        q.copy_(make(B, H * G, d))
        k1.copy_(make(B, H, d) * (1 + t % 5))
        v1.copy_(make(B, H, d))
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
        torch.cuda.synchronize()
        lens = [n + 1 for n in lens]
        assert rows.tolist() == lens
        for out, lse, window in zip(outs, lses, (0, 33)):
            for b in range(B):
                live = ref.seen_rows(lens[b] - 1, window, 4)
                for h in range(H):
                    s = slice(h * G, (h + 1) * G)
                    (kc, ks), (vc, vs) = c.held("k", b, h, lens[b]), c.held("v", b, h, lens[b])
                    check_unit(f64(q[b, s]), f64(out[b, s]), f64(lse[b, s]), kc[live], ks[live], vc[live], vs[live], d ** -0.5)
    assert skv.paged_status() == 0


def test_a_step_from_projections_over_codes():
    """Norm and rotation of a step's queries and keys, the keys written as codes, attention over them: near the same
    step over a bf16 cache, as far off as codes are (2^-4 of a key, 2^-4 of a value)."""
    H, G, d, n = 2, 4, 128, 200
    g = torch.Generator().manual_seed(12)
    make = lambda *s: torch.randn(s, generator=g).bfloat16().cuda()  # noqa: E731
    q, k, v = make(n, H * G, d), make(n, H, d), make(n, H, d)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    q2, k2 = skv.qk_norm_rope(q, k, pos, torch.empty_like(q), torch.empty_like(k))
    c = Codes([0], H, d, 16, 16, seed=1, cap=n)
    skv.paged_quantise(k2, v, c.k, c.v, c.ks, c.vs, c.table, c.lens, i32([0, n]))
    last = q2[-1:].contiguous()
    out, lse = torch.empty_like(last), torch.empty((1, H * G), device="cuda")
    skv.paged_attention(last, c.k, c.v, c.table, i32([n]), out, lse, k_scale=c.ks, v_scale=c.vs)
    for h in range(H):
        s = slice(h * G, (h + 1) * G)
        (kc, ks), (vc, vs) = c.held("k", 0, h, n), c.held("v", 0, h, n)
        check_unit(f64(last[0, s]), f64(out[0, s]), f64(lse[0, s]), kc, ks, vc, vs, d ** -0.5)
        for codes, size, x in ((kc, ks, k2), (vc, vs, v)):
            want = f64(x[:, h])
            assert (np.abs(codes * size[:, None] - want) <= np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * size[:, None])).all()


def test_two_streams_and_host_threads_over_codes():
    import threading
    c = Codes([9000, 500, 0, 3000], 2, 128, 16, 16, seed=18)
    qs = [ask(c, 4, 19 + i) for i in range(2)]
    want = [attend(c, q) for q in qs]
    torch.cuda.synchronize()
    got, failed = [[], []], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                got[i] = [attend(c, qs[i]) for _ in range(40)]
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
        assert len(got[i]) == 40 and all(torch.equal(o, want[i][0]) and torch.equal(s, want[i][1]) for o, s in got[i])


@pytest.mark.parametrize("d,ps,block,layout,lens,window,sink", [
    (128, 16, 8, "hnd", [1000, 33, 24, 7], 17, 20), (64, 8, 8, "nhd", [300, 31, 32, 33], 9, 1),
    (128, 8, 8, "hnd", [900, 50], 40, 3), (64, 64, 16, "hnd", [2000, 65], 300, 5), (128, 1024, 128, "nhd", [3000], 1000, 130)])
def test_codes_that_are_not_seen_may_be_anything(d, ps, block, layout, lens, window, sink):
    """NaN codes in every row that is not seen, NaN scales in every block without a row that is."""
    c = Codes(lens, 2, d, ps, block, layout, seed=d + ps)
    for b, n in enumerate(lens):
        live = ref.seen_rows(n - 1, window, sink)
        hidden = torch.as_tensor(np.setdiff1d(np.arange(n), live))
        page = c.table[b].cpu()[hidden // ps].long().cuda()
        for pool in (c.k, c.v):
            pool.view(torch.uint8)[page, :, (hidden % ps).cuda()] = 0x7F
        blocks = torch.as_tensor(np.setdiff1d(np.arange(-(-n // block)), live // block))
        page = c.table[b].cpu()[blocks * block // ps].long().cuda()
        for scale in (c.ks, c.vs):
            scale[page, :, (blocks * block % ps // block).cuda()] = math.nan
    q = ask(c, 4)
    for more in (0, 16384 // ps):
        c.cache["table"] = torch.cat([c.table, torch.full((len(lens), more), -1, dtype=torch.int32, device="cuda")], 1)
        check_codes(c, q, *attend(c, q, window=window, sink=sink), None, window, sink)
    assert skv.paged_status() == 0


def test_pools_of_codes_with_room_between_rows_and_pages():
    """Pools that are part of a larger tensor, and strides of dimensions that are never stepped through."""
    c = Codes([100, 37], 2, 64, 16, 16, seed=50)
    wide = [torch.full((c.k.shape[0], 3, 20, 128), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for w, pool in zip(wide, (c.k, c.v)):
        w[:, 1:, 2:18, 32:96] = pool.view(torch.uint8)
    pools = [w[:, 1:, 2:18, 32:96].view(E4M3) for w in wide]
    q = ask(c, 4)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    skv.paged_attention(q, *pools, c.table, c.lens, out, lse, k_scale=c.ks, v_scale=c.vs)
    check_codes(c, q, out, lse)
    x = torch.randn((5, 2, 64), device="cuda").to(torch.bfloat16)
    before = [w.clone() for w in wide]
    c.table = torch.cat([c.table, torch.full((2, 1), -1, dtype=torch.int32, device="cuda")], 1)
    skv.paged_quantise(x, x, *pools, c.ks, c.vs, c.table, i32([100, 37]), i32([0, 5, 5]))
    back = [torch.zeros_like(x) for _ in range(2)]
    skv.paged_dequantise(*pools, c.ks, c.vs, c.table, i32([105, 37]), i32([100, 0]), i32([0, 5, 5]), *back)
    for h in range(2):
        want, size = quantised(c, 0, h, "k", 100, f64(x[:, h]))
        assert np.array_equal(f64(back[0][:, h]), (want * size[:, None])[100:])
    for w, b in zip(wide, before):
        w[:, 1:, 2:18, 32:96] = b[:, 1:, 2:18, 32:96]
        assert torch.equal(w, b)
    assert skv.paged_status() == 0
    # one page, one head: their strides may be anything
    c = Codes([9], 1, 64, 16, 8, seed=51)
    pools = [p[int(c.table[0, 0])][None].as_strided((1, 1, 16, 64), (77, 33, 64, 1)) for p in (c.k, c.v)]
    scales = [s[int(c.table[0, 0])][None] for s in (c.ks, c.vs)]
    q = ask(c, 2)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    skv.paged_attention(q, *pools, torch.zeros((1, 1), dtype=torch.int32, device="cuda"), c.lens, out, lse, k_scale=scales[0],
                        v_scale=scales[1])
    check_codes(c, q, out, lse)


def test_pools_of_codes_that_are_expanded_are_refused():
    c = Codes([9], 1, 64, 16, 8, seed=52)
    q = ask(c, 2)
    for dim, shape in ((1, (-1, 2, -1, -1)), (0, (6, -1, -1, -1))):
        pools = [p[:1].expand(*shape) if dim == 0 else p.expand(*shape) for p in (c.k, c.v)]
        scales = [torch.ones((pools[0].shape[0], pools[0].shape[1], 2), device="cuda") for _ in range(2)]
        heads = 2 * pools[0].shape[1]
        with pytest.raises(skv.ShadowKVError) as e:
            skv.paged_attention(q[:, :1].expand(-1, heads, -1).contiguous(), *pools, c.table, c.lens,
                                torch.empty((1, heads, 64), dtype=torch.bfloat16, device="cuda"), k_scale=scales[0], v_scale=scales[1])
        assert e.value.code == -1
