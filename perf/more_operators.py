"""Cases of the paged cache's further operators, for measuring them: a plain form of each in elementary torch
operations, the framework's own calls, and the definition in 64 bits.

The operators (all on one GPU; b sequences, n_q query heads over H key/value heads, G = n_q / H, head
dim d, a cache of pages of ps rows with a page table; an 8-bit cache holds e4m3 codes and an fp32
scale for every block of `block` rows of a page and head, a value being code * scale):

* quantise: the new keys and values of every sequence, tokens start[b] .. start[b+1], become its rows
  lens[b] on of an 8-bit cache.  A block's scale is the smallest power of two 2^e, e >= -100, with
  |x| <= 448 * 2^e for the finite x among its new rows; where the block holds rows of the sequence
  already, its old scale if that is larger, and if it is not, the held codes are rounded again to the new one.
* dequantise: rows first[b] on of every sequence are read back, into tokens start[b] .. start[b+1].
* attend: one new token per sequence, softmax(scale q.K^T).V with the log-sum-exp over the rows j with
  j < sink or j >= lens[b] - window (window 0: over all), over an 8-bit cache or one of the other types.
* prompt: the same for many new tokens per sequence; token start[b] + i is row r = lens[b] - n_b + i
  (n_b = start[b+1] - start[b]) and sees rows j <= r with j < sink or j > r - window.
"""
import math

import numpy as np
import torch

own = False


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of 8 sequences (the 128K batch-8 decode workload): a row each, into blocks that hold some
        dict(name="quantise step b8", op="quantise", wide="bf16", layout="hnd", batch=8, tokens=1, ragged=False, n_kv=8,
             d=128, ps=16, block=16),
        # a 32K prompt's keys and values
        dict(name="quantise prompt 32K", op="quantise", wide="bf16", layout="hnd", batch=1, tokens=32768, ragged=False,
             n_kv=8, d=128, ps=64, block=64),
        # prompts of several requests of a small fp32 model, token-major pages
        dict(name="quantise ragged fp32", op="quantise", wide="f32", layout="nhd", batch=12, tokens=1021, ragged=True,
             n_kv=2, d=64, ps=32, block=8),
        # whole 32K contexts read back for a layer that wants them in bf16
        dict(name="dequantise 32K b4", op="dequantise", wide="bf16", layout="hnd", batch=4, tokens=32768, ragged=False,
             n_kv=8, d=128, ps=16, block=16),
        # the last rows of a few requests, in fp32
        dict(name="dequantise ragged fp32", op="dequantise", wide="f32", layout="nhd", batch=5, tokens=613, ragged=True,
             n_kv=2, d=64, ps=64, block=32),
        # one short conversation over an 8-bit cache: the latency of a step
        dict(name="attend 1K b1 8-bit", op="attend", kind="q8", layout="hnd", batch=1, len=1013, ragged=False, n_q=32,
             n_kv=8, d=128, ps=16, block=16, window=0, sink=0),
        # the 128K batch-8 decode workload with whole 8-bit caches
        dict(name="attend 128K b8 8-bit", op="attend", kind="q8", layout="hnd", batch=8, len=131072, ragged=False, n_q=32,
             n_kv=8, d=128, ps=64, block=64, window=0, sink=0),
        # many conversations, 8-bit token-major pages, the last 1000 rows and four first ones visible
        dict(name="attend b192 8-bit window", op="attend", kind="q8", layout="nhd", batch=192, len=4097, ragged=True,
             n_q=32, n_kv=4, d=128, ps=32, block=16, window=1000, sink=4),
        # 128K contexts in bf16 of which a layer sees 4096 rows and four first ones
        dict(name="attend 128K b8 window", op="attend", kind="bf16", layout="hnd", batch=8, len=131072, ragged=True, n_q=32,
             n_kv=8, d=128, ps=16, window=4096, sink=4),
        # a few drafted tokens of each of 8 conversations checked at once
        dict(name="prompt drafts b8", op="prompt", layout="hnd", batch=8, len=4099, tokens=5, ragged=True, n_q=32, n_kv=8,
             d=128, ps=16, window=0, sink=0),
        # chunks of several long prompts in a layer with a window
        dict(name="prompt chunks window", op="prompt", layout="nhd", batch=6, len=16384, tokens=4093, ragged=True, n_q=32,
             n_kv=8, d=128, ps=64, window=1024, sink=4),
        # a whole 32K prompt: the largest
        dict(name="prompt 32K", op="prompt", layout="hnd", batch=1, len=32768, tokens=32768, ragged=False, n_q=32, n_kv=8,
             d=128, ps=16, window=0, sink=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantise", "dequantise", "attend", "attend", "prompt", "prompt"])
    c = dict(op=op, layout=rng.choice(["hnd", "nhd"]), n_kv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 128, 128]),
             ps=rng.choice([8, 16, 32, 64, 128]), ragged=rng.random() < 0.7)
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    if op in ("quantise", "dequantise"):
        c.update(wide=rng.choice(["bf16", "bf16", "f32"]), batch=_log(rng, 1, 64),
                 block=rng.choice([x for x in (8, 16, 32, 64, 128) if x <= c["ps"]]))
        room = 131072 * 8 * 128 * 3 // (c["n_kv"] * c["d"] * (5 if c["wide"] == "f32" else 3))
        c["tokens"] = _log(rng, 1, max(1, min(32768, room // c["batch"])))
        return c
    c["sink"] = rng.choice([0, 0, 1, 4, rng.randint(0, 200)])
    if op == "attend":
        c.update(kind=rng.choice(["q8", "q8", "q8", "bf16", "fp8", "f32"]), batch=_log(rng, 1, 256), n_q=c["n_kv"] * group)
        if c["kind"] == "q8":
            c["block"] = rng.choice([x for x in (8, 16, 32, 64, 128) if x <= c["ps"]])
        row = c["n_kv"] * c["d"] * {"bf16": 4, "fp8": 3, "f32": 8, "q8": 2}[c["kind"]]
        c["len"] = _log(rng, 1, max(1, min(262144, (1 << 31) // (row * c["batch"]))))
        c["window"] = 0 if c["kind"] == "q8" and rng.random() < 0.5 else _log(rng, 1, 16384)
        return c
    c.update(batch=_log(rng, 1, 24), n_q=c["n_kv"] * group)
    # pairs of a token and a row that it sees: a quarter of the largest listed case's at most
    pairs = 32 * 32768 * 32768 // 8 // c["n_q"]
    c["len"] = _log(rng, 1, 32768)
    c["tokens"] = _log(rng, 1, max(1, min(c["len"], pairs // (c["len"] * c["batch"]))))
    c["window"] = rng.choice([0, _log(rng, 1, 16384)])
    if c["window"] == 0:
        c["sink"] = 0
    return c


def _spread(n, c, k):
    """Sizes of the sequences: all alike, or spread over [0, n] by a golden ratio with the largest first."""
    if not c["ragged"]:
        return [n] * c["batch"]
    return [n] + [int(n * ((i * k) % 1.0)) for i in range(1, c["batch"])]


def _tokens(c):
    return _spread(c["tokens"], c, 0.6180339887498949)


def _lens(c):
    """Rows of the sequences, in a prompt those of its tokens among them."""
    lens = _spread(c["len"], c, 0.7548776662466927 if c["op"] == "prompt" else 0.6180339887498949)
    return [max(a, n) for a, n in zip(lens, _tokens(c))] if c["op"] == "prompt" else lens


def _held(c):
    """Rows that the sequences hold before new ones are written, or that stand before those read back."""
    return [(i * 331 + 5) % 1999 for i in range(c["batch"])]


def _seen(c, r):
    """How many rows the token that is row r sees, counts for an array of rows."""
    r = np.asarray(r, dtype=np.int64)
    if c["window"] == 0:
        return r + 1
    near = np.minimum(r + 1, c["window"])
    return near + np.minimum(c["sink"], r + 1 - near)


def _types(c):
    wide = torch.float32 if c["kind"] == "f32" else torch.bfloat16
    val = torch.float8_e5m2 if c["kind"] == "fp8" else wide
    return (torch.float8_e4m3fn, torch.float8_e4m3fn) if c["kind"] == "q8" else (wide, val)


def work(c):
    d, H = c["d"], c["n_kv"]
    if c["op"] in ("quantise", "dequantise"):
        n = sum(_tokens(c))
        es = 4 if c["wide"] == "f32" else 2
        if c["op"] == "quantise":
            blocks = sum(-(-(a + n) // c["block"]) - a // c["block"] for a, n in zip(_held(c), _tokens(c)) if n)
        else:
            blocks = n // c["block"]
        return {"bytes": n * H * d * 2 * (es + 1) + 8 * H * blocks, "flops": n * H * d * 4}
    heads = c["n_q"]
    if c["op"] == "attend":
        lens = _lens(c)
        key, val = (t.itemsize for t in _types(c))
        seen = int(sum(_seen(c, n - 1) for n in lens if n))
        q = c["batch"] * heads
        scales = 8 * H * seen // c["block"] if c["kind"] == "q8" else 0
        return {"bytes": seen * H * d * (key + val) + scales + 2 * q * d * (4 if c["kind"] == "f32" else 2) + 4 * q,
                "flops": 4 * d * seen * heads}
    pairs = rows = n_all = 0
    for a, n in zip(_lens(c), _tokens(c)):
        if n:
            pairs += int(_seen(c, np.arange(a - n, a)).sum())
            rows += a if c["window"] == 0 else min(a, n + c["window"] - 1 + c["sink"])
            n_all += n
    return {"bytes": rows * H * d * 4 + n_all * heads * (4 * d + 4), "flops": 4 * d * pairs * heads}


# ------------------------------------------------------------------ inputs

def _pool(c, gen, pages, dtype):
    """Rows of a few heavy dimensions, as keys and values have them."""
    shape = (pages, c["n_kv"], c["ps"], c["d"]) if c["layout"] == "hnd" else (pages, c["ps"], c["n_kv"], c["d"])
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32 if dtype == torch.float32 else torch.bfloat16)
    if dtype == torch.float8_e4m3fn:
        x = x * 112.0                        # codes that use their block's range
        x = x.clamp(-448.0, 448.0)
    x = x.to(dtype)
    return x if c["layout"] == "hnd" else x.permute(0, 2, 1, 3)


def _scales(c, gen, pages, size):
    """Powers of two around size / 112."""
    e = torch.randint(-2, 2, (pages, c["n_kv"], c["ps"] // c["block"]), generator=gen, device="cuda")
    return torch.exp2(e.float() + round(math.log2(size / 112.0)))


def _table(c, gen, lens, cap):
    """Page ids of every sequence in random order over the pool, -1 where a sequence has no page."""
    width = max(1, -(-cap // c["ps"]))
    need = torch.tensor([-(-n // c["ps"]) for n in lens], device="cuda")
    total = int(sum(-(-n // c["ps"]) for n in lens))
    pages = total + 3
    table = torch.full((c["batch"], width), -1, device="cuda", dtype=torch.int32)
    used = torch.arange(width, device="cuda")[None] < need[:, None]
    table[used] = torch.randperm(pages, generator=gen, device="cuda")[:total].to(torch.int32)
    return table, pages


def _i32(x):
    return torch.tensor(x, device="cuda", dtype=torch.int32)


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": c}
    if c["op"] in ("quantise", "dequantise"):
        n, held = _tokens(c), _held(c)
        lens = [a + b for a, b in zip(held, n)]
        s["table"], pages = _table(c, gen, lens, max(lens))
        s["k_cache"] = _pool(c, gen, pages, torch.float8_e4m3fn)
        s["v_cache"] = _pool(c, gen, pages, torch.float8_e4m3fn)
        s["k_scale"], s["v_scale"] = _scales(c, gen, pages, 1.0), _scales(c, gen, pages, 1.0)
        s["start"] = _i32(np.concatenate([[0], np.cumsum(n)]))
        s["lens"] = _i32(held if c["op"] == "quantise" else lens)
        wide = torch.float32 if c["wide"] == "f32" else torch.bfloat16
        shape = (sum(n), c["n_kv"], c["d"])
        if c["op"] == "dequantise":
            s["first"] = _i32(held)
            s["k_out"], s["v_out"] = (torch.zeros(shape, device="cuda", dtype=wide) for _ in range(2))
            return s
        # keys of tokens of different weight with a few heavy dimensions, out of a fused projection; values
        fused = torch.randn((sum(n), 2 * c["n_kv"] * c["d"]), generator=gen, device="cuda", dtype=wide)
        s["k"] = fused[:, :c["n_kv"] * c["d"]].unflatten(1, shape[1:])
        s["v"] = fused[:, c["n_kv"] * c["d"]:].unflatten(1, shape[1:])
        s["k"] *= torch.randn((sum(n), 1, 1), generator=gen, device="cuda").mul_(0.7).exp2_().to(wide)
        s["k"][..., 3::32] *= 6
        return s
    lens = _lens(c)
    s["lens"] = _i32(lens)
    s["table"], pages = _table(c, gen, lens, max(lens))
    key, val = _types(c) if c["op"] == "attend" else (torch.bfloat16, torch.bfloat16)
    s["k_cache"], s["v_cache"] = _pool(c, gen, pages, key), _pool(c, gen, pages, val)
    if key == torch.float8_e4m3fn:
        s["k_scale"], s["v_scale"] = _scales(c, gen, pages, 1.0), _scales(c, gen, pages, 1.0)
    if c["op"] == "prompt":
        s["start"] = _i32(np.concatenate([[0], np.cumsum(_tokens(c))]))
    rows = c["batch"] if c["op"] == "attend" else sum(_tokens(c))
    wide = torch.float32 if key == torch.float32 else torch.bfloat16
    q = torch.randn((rows, c["n_q"], c["d"]), generator=gen, device="cuda", dtype=wide)
    s["q"] = q * torch.linspace(0.5, 3.0, c["n_q"], device="cuda")[None, :, None].to(wide)   # flat and peaked heads
    s["out"] = torch.zeros_like(q)
    s["lse"] = torch.zeros((rows, c["n_q"]), device="cuda")
    return s


# ------------------------------------------------------------------ plain forms

def _bytes(x):
    return x.view(torch.uint8) if x.dtype in (torch.float8_e5m2, torch.float8_e4m3fn) else x


def _places(s, first):
    """Sequence and row of every token."""
    n = (s["start"][1:] - s["start"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(len(n), device="cuda"), n)
    return seq, torch.arange(len(seq), device="cuda") - s["start"][seq] + first[seq]


def _plain_quantise(s):
    c = s["case"]
    ps, block, nb = c["ps"], c["block"], c["ps"] // c["block"]
    seq, row = _places(s, s["lens"])
    page, at = s["table"][seq, row // ps].long(), row % ps
    place = page * nb + at // block                                     # a token's block among all blocks
    # the block that a sequence's first new row joins, and the rows that it holds
    lens, n = s["lens"].long(), s["start"][1:] - s["start"][:-1]
    b = ((lens % block != 0) & (n > 0)).nonzero().flatten()
    held = lens[b] // block * block
    j_page, j_at = s["table"][b, held // ps].long(), held % ps
    joined = j_page * nb + j_at // block
    offset = torch.arange(block, device="cuda")
    inside = (held[:, None] + offset < lens[b][:, None])[:, None, :, None]           # [joined][1][block][1]
    for x, cache, scale in ((s["k"], s["k_cache"], s["k_scale"]), (s["v"], s["v_cache"], s["v_scale"])):
        x = x.float()
        x = torch.where(x.isfinite(), x, math.nan)
        most = torch.zeros((scale.shape[0] * nb, c["n_kv"]), device="cuda")
        most.scatter_reduce_(0, place[:, None].expand(-1, c["n_kv"]), x.abs().nan_to_num(0.0).amax(-1), "amax")
        part, e = torch.frexp(most)                                     # most = part 2^e, part in [0.5, 1)
        new = torch.exp2((e - torch.where(part <= 0.875, 9, 8)).clamp(min=-100).float())
        old = scale.transpose(1, 2).reshape(-1, c["n_kv"])
        new[joined] = torch.maximum(new[joined], old[joined])
        rows = (j_page[:, None], slice(None), j_at[:, None] + offset)
        codes = _bytes(cache)[rows].view(torch.float8_e4m3fn).transpose(1, 2)         # [joined][H][block][d]
        again = (codes.float() * (old[joined] / new[joined])[..., None, None]).to(torch.float8_e4m3fn)
        again = torch.where(inside, _bytes(again), _bytes(codes))
        _bytes(cache)[rows] = again.transpose(1, 2)
        _bytes(cache)[page, :, at] = _bytes((x / new[place][..., None]).to(torch.float8_e4m3fn))
        scale[page, :, at // block] = new[place]
    return _quantise_outputs(s)


def _quantise_outputs(s):
    return {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}


def _plain_dequantise(s):
    c = s["case"]
    seq, row = _places(s, s["first"])
    page, at = s["table"][seq, row // c["ps"]].long(), row % c["ps"]
    for name in ("k", "v"):
        codes = _bytes(s[name + "_cache"])[page, :, at].view(torch.float8_e4m3fn).float()
        s[name + "_out"].copy_(codes * s[name + "_scale"][page, :, at // c["block"]][..., None])
    return {"k_out": s["k_out"], "v_out": s["v_out"]}


def _rows(s, name, page):
    """Rows of whole pages as numbers, [..][H][rows][d] of a table [..][pages]."""
    c = s["case"]
    x = _bytes(s[name + "_cache"])[page].view(s[name + "_cache"].dtype).float()
    if name + "_scale" in s:
        x = x * s[name + "_scale"][page].repeat_interleave(c["block"], -1)[..., None]
    return x.transpose(-4, -3).flatten(-3, -2)


def _plain_attend(s):
    c = s["case"]
    nk, d, g = c["n_kv"], c["d"], c["n_q"] // c["n_kv"]
    # as many sequences at a time as leave room for their rows in 32 bits
    step = max(1, (1 << 33) // (s["table"].shape[1] * c["ps"] * nk * d))
    for lo in range(0, c["batch"], step):
        lens, page = s["lens"][lo:lo + step, None], s["table"][lo:lo + step].clamp(min=0).long()
        j = torch.arange(page.shape[1] * c["ps"], device="cuda")[None]
        seen = j < lens
        if c["window"]:
            seen = seen & ((j < c["sink"]) | (j >= lens - c["window"]))
        z = torch.matmul(s["q"][lo:lo + step].float().unflatten(1, (nk, g)), _rows(s, "k", page).transpose(-1, -2)) / math.sqrt(d)
        z = z.masked_fill(~seen[:, None, None], -math.inf)
        top = z.amax(-1, keepdim=True).clamp(min=-1e30)
        z = torch.exp(z - top)
        total = z.sum(-1, keepdim=True)
        v = _rows(s, "v", page).masked_fill(~seen[:, None, :, None], 0.0)
        o = torch.matmul(z / torch.where(total == 0, 1.0, total), v)
        s["out"][lo:lo + step] = o.flatten(1, 2).to(s["out"].dtype)
        s["lse"][lo:lo + step] = torch.where(total == 0, -math.inf, top + torch.log(total)).flatten(1)
        del z, v
    return {"out": s["out"], "lse": s["lse"]}


def _plain_prompt(s):
    c = s["case"]
    nk, d, g = c["n_kv"], c["d"], c["n_q"] // c["n_kv"]
    start, lens = s["start"].tolist(), s["lens"].tolist()
    step = max(1, 512 * 32 // c["n_q"])
    for b in range(c["batch"]):
        n = start[b + 1] - start[b]
        if n == 0:
            continue
        page = s["table"][b, :-(-lens[b] // c["ps"])].long()
        k, v = _rows(s, "k", page), _rows(s, "v", page)                               # [H][rows][d]
        for lo in range(0, n, step):
            hi = min(n, lo + step)
            r = torch.arange(lens[b] - n + lo, lens[b] - n + hi, device="cuda")[:, None]
            stop = lens[b] - n + hi                                                   # rows behind are seen by none
            j = torch.arange(stop, device="cuda")[None]
            seen = j <= r
            if c["window"]:
                seen = seen & ((j < c["sink"]) | (j > r - c["window"]))
            at = slice(start[b] + lo, start[b] + hi)
            q = s["q"][at].float().unflatten(1, (nk, g)).permute(1, 2, 0, 3)          # [H][G][tokens][d]
            z = torch.matmul(q, k[:, None, :stop].transpose(-1, -2)) / math.sqrt(d)
            z.masked_fill_(~seen, -math.inf)
            top = z.amax(-1, keepdim=True)
            z.sub_(top).exp_()
            total = z.sum(-1, keepdim=True)
            o = torch.matmul(z, v[:, None, :stop]) / total
            s["out"][at] = o.permute(2, 0, 1, 3).flatten(1, 2).to(s["out"].dtype)
            s["lse"][at] = (top + torch.log(total))[..., 0].permute(2, 0, 1).flatten(1)
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------ one pass

def run(s):
    c = s["case"]
    if not own:
        return {"quantise": _plain_quantise, "dequantise": _plain_dequantise, "attend": _plain_attend,
                "prompt": _plain_prompt}[c["op"]](s)
    import sparse_kv_cache_gb300 as skv
    if c["op"] == "quantise":
        skv.paged_quantise(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["lens"],
                           s["start"])
        return _quantise_outputs(s)
    if c["op"] == "dequantise":
        skv.paged_dequantise(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["lens"], s["first"],
                             s["start"], s["k_out"], s["v_out"])
        return {"k_out": s["k_out"], "v_out": s["v_out"]}
    if c["op"] == "attend":
        scales = dict(k_scale=s["k_scale"], v_scale=s["v_scale"]) if c["kind"] == "q8" else {}
        skv.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["out"], lse=s["lse"],
                            window=c["window"], sink=c["sink"], **scales)
    else:
        skv.paged_prompt_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["start"], s["out"],
                                   lse=s["lse"], window=c["window"], sink=c["sink"])
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] in ("attend", "prompt") and work(c)["flops"] > 4e12:
        return None
    return {"quantise": _exact_quantise, "dequantise": _exact_dequantise, "attend": _exact_attend,
            "prompt": _exact_prompt}[c["op"]](s)


def _e4m3(x):
    """Nearest e4m3 numbers, ties to even, of |x| <= 448."""
    grid = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(x), 1e-300))), -6.0) - 3.0)
    return np.rint(x / grid) * grid


def _exact_quantise(s):
    """Block by block on the host."""
    c = s["case"]
    H, ps, block = c["n_kv"], c["ps"], c["block"]
    table, start, lens = (s[n].cpu().numpy().astype(np.int64) for n in ("table", "start", "lens"))
    got = {}
    for name in ("k", "v"):
        x = s[name].double().cpu().numpy()
        cache, scale = s[name + "_cache"].cpu().float().double().numpy(), s[name + "_scale"].double().cpu().numpy()
        for b in range(c["batch"]):
            row, end = int(lens[b]), int(lens[b] + start[b + 1] - start[b])
            while row < end:
                lo = row // block * block
                hi = min(end, lo + block)
                page, at = table[b, lo // ps], lo % ps
                new = x[start[b] + row - lens[b]:start[b] + hi - lens[b]]              # [rows][H][d]
                most = np.abs(new).max((0, 2))
                size = np.exp2(np.maximum(np.ceil(np.log2(np.maximum(most, 1e-300) / 448.0)), -100.0))
                if row > lo:
                    was = scale[page, :, at // block]
                    size = np.maximum(size, was)
                    cache[page, :, at:at + row - lo] = _e4m3(cache[page, :, at:at + row - lo] * (was / size)[:, None, None])
                scale[page, :, at // block] = size
                cache[page, :, at + row - lo:at + hi - lo] = _e4m3(new / size[:, None]).transpose(1, 0, 2)
                row = hi
        got[name + "_cache"], got[name + "_scale"] = torch.from_numpy(cache), torch.from_numpy(scale)
    return got


def _exact_dequantise(s):
    c = s["case"]
    start, first = s["start"].tolist(), s["first"].tolist()
    got = {}
    for name in ("k", "v"):
        out = torch.zeros(s[name + "_out"].shape, dtype=torch.float64, device="cuda")
        for b in range(c["batch"]):
            at = torch.arange(first[b], first[b] + start[b + 1] - start[b], device="cuda")
            page = s["table"][b, at // c["ps"]].long()
            codes = s[name + "_cache"].view(torch.uint8)[page, :, at % c["ps"]].view(torch.float8_e4m3fn)
            out[start[b]:start[b + 1]] = codes.double() * s[name + "_scale"].double()[page, :, at % c["ps"] // c["block"], None]
        got[name + "_out"] = out
    return got


def _unit(s, name, b, h, rows):
    """The given rows of a unit."""
    c = s["case"]
    page, at = s["table"][b, rows // c["ps"]].long(), rows % c["ps"]
    cache = s[name + "_cache"]
    x = (cache.view(torch.uint8)[page, h, at].view(cache.dtype) if cache.dtype.itemsize == 1 else cache[page, h, at]).double()
    return x * s[name + "_scale"][page, h, at // c["block"], None].double() if name + "_scale" in s else x


def _exact_attend(s):
    c = s["case"]
    g = c["n_q"] // c["n_kv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        near = max(0, n - c["window"]) if c["window"] else 0
        rows = torch.cat([torch.arange(min(c["sink"], near)), torch.arange(near, n)]).cuda()
        if n == 0:
            continue
        for h in range(c["n_kv"]):
            heads = slice(h * g, (h + 1) * g)
            z = (s["q"][b, heads].double() @ _unit(s, "k", b, h, rows).T) * c["d"] ** -0.5
            lse[b, heads] = z.logsumexp(-1)
            out[b, heads] = (z - lse[b, heads, None]).exp() @ _unit(s, "v", b, h, rows)
    return {"out": out, "lse": lse}


def _exact_prompt(s):
    c = s["case"]
    g = c["n_q"] // c["n_kv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    start = s["start"].tolist()
    for b, n in enumerate(s["lens"].tolist()):
        first = n - (start[b + 1] - start[b])
        rows = torch.arange(n, device="cuda")
        for h in range(c["n_kv"]):
            if first == n:
                break
            k, v = _unit(s, "k", b, h, rows), _unit(s, "v", b, h, rows)
            heads = slice(h * g, (h + 1) * g)
            for lo in range(first, n, 1024):
                r = rows[lo:min(n, lo + 1024)]
                hi = int(r[-1]) + 1
                at = slice(start[b] + lo - first, start[b] + hi - first)
                away = r[:, None] - rows[None, :hi]                                   # how far back a row lies
                hidden = (away < 0) | ((away >= c["window"]) & (rows[None, :hi] >= c["sink"]) & (c["window"] > 0))
                z = torch.einsum("tgd,jd->gtj", s["q"][at, heads].double(), k[:hi]) * c["d"] ** -0.5
                z = z.masked_fill(hidden, -math.inf)
                total = z.logsumexp(-1)
                lse[at, heads] = total.T
                out[at, heads] = torch.einsum("gtj,jd->tgd", (z - total[..., None]).exp(), v[:hi])
    return {"out": out, "lse": lse}
