"""Cases of the paged-cache operators, for measuring them: a plain form of each in elementary torch
operations, the framework's own calls, and the definition in 64 bits.

The operators (all on one GPU; T tokens, b sequences, n_q query heads over H key/value heads,
G = n_q / H, head dim d, a cache of pages of ps rows with a page table):

* norm: per head x <- x / sqrt(mean(x^2) + eps) * w, then the rotary position of the token
  (half-split pairs, theta_i = base^(-2i/rd)), for q and k of every token; k and v are written into
  their sequence's rows of the paged cache in the same pass, with the row's position and a weight of
  zero where the cache keeps them.
* attend: one new token per sequence over its paged cache, softmax(scale q.K^T).V with the
  log-sum-exp; where asked, the weight that each cached row received is added to a running sum.
* evict: per (sequence, KV head) the cache is brought down to `budget` rows: the `recent` last
  positions, the first `sink` positions, and the heaviest of the rest stay; every kept row behind the
  budget moves into a row that was given up, in ascending order of both.
"""
import math

import numpy as np
import torch

own = False

BASE = 500000.0
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of 8 sequences (the 128K batch-8 decode workload): latency of a small launch
        dict(name="norm step b8", op="norm", kind="bf16", layout="hnd", batch=8, tokens=1, n_q=32, n_kv=8, d=128,
             rd=128, ps=16, pad=0, track=True, k_out=False),
        # a 32K prompt's queries and keys out of a fused projection, keys also handed on whole
        dict(name="norm prompt 32K", op="norm", kind="bf16", layout="hnd", batch=1, tokens=32768, n_q=32, n_kv=8,
             d=128, rd=128, ps=16, pad=0, track=False, k_out=True),
        # prompts of several requests in one padded batch, e5m2 values, token-major pages, half of each head rotated
        dict(name="norm padded fp8", op="norm", kind="fp8", layout="nhd", batch=5, tokens=1021, n_q=16, n_kv=2, d=128,
             rd=64, ps=64, pad=37, track=False, k_out=False),
        # one short conversation: the latency of a single decode step
        dict(name="attend 1K b1", op="attend", kind="bf16", layout="hnd", batch=1, len=1013, ragged=False, n_q=32, n_kv=8,
             d=128, ps=16, weigh=False),
        # many short conversations of very different lengths, some slots idle
        dict(name="attend short b192", op="attend", kind="bf16", layout="nhd", batch=192, len=611, ragged=True, n_q=32,
             n_kv=4, d=128, ps=32, weigh=False),
        # the 32K batch-4 decode workload
        dict(name="attend 32K b4", op="attend", kind="bf16", layout="hnd", batch=4, len=32768, ragged=False, n_q=32,
             n_kv=8, d=128, ps=16, weigh=False),
        # the 128K batch-8 decode workload with whole caches: the largest
        dict(name="attend 128K b8", op="attend", kind="bf16", layout="hnd", batch=8, len=131072, ragged=False, n_q=32,
             n_kv=8, d=128, ps=64, weigh=False),
        # 64K contexts with e5m2 values
        dict(name="attend 64K b8 fp8", op="attend", kind="fp8", layout="hnd", batch=8, len=65536, ragged=True, n_q=32,
             n_kv=8, d=128, ps=16, weigh=False),
        # a small fp32 model
        dict(name="attend 4K fp32", op="attend", kind="f32", layout="hnd", batch=3, len=4099, ragged=True, n_q=8, n_kv=2,
             d=64, ps=8, weigh=False),
        # 64K contexts that also keep each row's accumulated weight for eviction
        dict(name="weigh 64K b4", op="attend", kind="bf16", layout="hnd", batch=4, len=65536, ragged=True, n_q=32, n_kv=8,
             d=128, ps=16, weigh=True),
        # a decode step over its budget by one row in every head
        dict(name="evict one b8", op="evict", kind="bf16", layout="hnd", batch=8, len=2081, ragged=False, n_kv=8, d=128,
             ps=16, budget=2080, recent=32, sink=4),
        # a 128K prompt brought down to the sparse budget
        dict(name="evict 128K b8", op="evict", kind="bf16", layout="hnd", batch=8, len=131072, ragged=True, n_kv=8, d=128,
             ps=16, budget=2464, recent=32, sink=4),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "attend", "attend", "evict"])
    c = dict(op=op, kind=rng.choice(["bf16", "bf16", "fp8", "f32"]), layout=rng.choice(["hnd", "nhd"]),
             n_kv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 128, 128]), ps=rng.choice([8, 16, 32, 64, 128]))
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    if op == "norm":
        c.update(batch=_log(rng, 1, 64), n_q=c["n_kv"] * group, rd=rng.choice([c["d"], c["d"], c["d"] // 2]),
                 track=rng.random() < 0.5, k_out=rng.random() < 0.5)
        room = 32768 * 48 * 128 * 2 // ((c["n_q"] + 3 * c["n_kv"]) * c["d"] * (4 if c["kind"] == "f32" else 2))
        c["tokens"] = _log(rng, 1, max(1, min(32768, room // c["batch"])))
        c["pad"] = rng.choice([0, 0, rng.randint(1, 40)])
        return c
    c["batch"] = _log(rng, 1, 256)
    row = c["n_kv"] * c["d"] * {"bf16": 4, "fp8": 3, "f32": 8}[c["kind"]]
    most = 1 << 31 if op == "attend" else 1 << 30          # half of the largest listed cache at most
    c["len"] = _log(rng, 1, max(1, min(262144, most // (row * c["batch"]))))
    c["ragged"] = rng.random() < 0.7
    if op == "attend":
        c.update(n_q=c["n_kv"] * group, weigh=rng.random() < 0.3)
    else:
        budget = _log(rng, 1, max(1, min(8192, c["len"])))
        recent = rng.randint(0, min(64, budget))
        c.update(budget=budget, recent=recent, sink=rng.randint(0, min(8, budget - recent)))
    return c


def _lens(c):
    """Lengths of the sequences: all alike, or spread over [0, len] by the golden ratio with the longest first."""
    if not c["ragged"]:
        return [c["len"]] * c["batch"]
    return [c["len"]] + [int(c["len"] * ((i * 0.6180339887498949) % 1.0)) for i in range(1, c["batch"])]


def _types(c):
    wide = torch.float32 if c["kind"] == "f32" else torch.bfloat16
    return wide, torch.float8_e5m2 if c["kind"] == "fp8" else wide


def work(c):
    wide, val = _types(c)
    es, ev, d = wide.itemsize, val.itemsize, c["d"]
    if c["op"] == "norm":
        n = c["batch"] * c["tokens"]
        read = (c["n_q"] + 2 * c["n_kv"]) * d * es + 12
        write = (c["n_q"] + c["n_kv"] * (2 if c["k_out"] else 1)) * d * es + c["n_kv"] * d * ev + (8 * c["n_kv"] if c["track"] else 0)
        return {"bytes": n * (read + write), "flops": n * (c["n_q"] + c["n_kv"]) * d * 8}
    lens = _lens(c)
    if c["op"] == "attend":
        rows = sum(lens) * c["n_kv"]
        heads = c["batch"] * c["n_q"]
        table = 4 * sum(-(-n // c["ps"]) for n in lens)
        return {"bytes": rows * d * (es + ev) + (8 * rows if c["weigh"] else 0) + 2 * heads * d * es + 4 * heads + table,
                "flops": 4 * d * sum(lens) * c["n_q"]}
    n_in = sum(n for n in lens) * c["n_kv"]
    kept = sum(min(n, c["budget"]) for n in lens) * c["n_kv"]
    # rows that have to move: the kept ones expected behind the budget, were every row as likely to be kept
    moved = sum(c["budget"] * (n - c["budget"]) / n for n in lens if n > c["budget"]) * c["n_kv"]
    return {"bytes": 8 * n_in + 8 * kept + 2 * moved * d * (es + ev), "flops": 4 * n_in}


# ------------------------------------------------------------------ inputs

def _pool(c, gen, pages):
    wide, val = _types(c)
    shape = (pages, c["n_kv"], c["ps"], c["d"]) if c["layout"] == "hnd" else (pages, c["ps"], c["n_kv"], c["d"])
    out = []
    for t in (wide, val):
        x = torch.randn(shape, generator=gen, device="cuda", dtype=wide)
        out.append((x if c["layout"] == "hnd" else x.permute(0, 2, 1, 3)) if t is wide
                   else (x.to(t) if c["layout"] == "hnd" else x.to(t).permute(0, 2, 1, 3)))
    return out


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


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    wide, _ = _types(c)
    s = {"case": c}
    if c["op"] == "norm":
        b, n, nq, nk, d = c["batch"], c["tokens"], c["n_q"], c["n_kv"], c["d"]
        rows = b * n
        start = [(i * 331) % 1999 for i in range(b)]                       # rows that each sequence holds already
        s["table"], pages = _table(c, gen, [x + n for x in start], 1999 + n)
        s["k_cache"], s["v_cache"] = _pool(c, gen, pages)
        qkv = torch.randn((rows + c["pad"], (nq + 2 * nk) * d), generator=gen, device="cuda", dtype=wide)
        s["q"] = qkv[:, :nq * d].unflatten(1, (nq, d))
        s["k"] = qkv[:, nq * d:(nq + nk) * d].unflatten(1, (nk, d))
        s["v"] = qkv[:, (nq + nk) * d:].unflatten(1, (nk, d))
        s["q_weight"] = 1 + 0.2 * torch.randn(d, generator=gen, device="cuda", dtype=wide)
        s["k_weight"] = 1 + 0.2 * torch.randn(d, generator=gen, device="cuda", dtype=wide)
        at = torch.tensor(start, device="cuda")[:, None] + torch.arange(n, device="cuda")[None]
        off = torch.randint(0, 1 << 17, (b, 1), generator=gen, device="cuda")     # evicted caches: position >= row
        tail = torch.full((c["pad"],), -1, device="cuda", dtype=torch.int32)      # padding behind the last sequence
        s["index"] = torch.cat([at.flatten().to(torch.int32), tail])
        s["positions"] = torch.cat([(at + off).flatten().to(torch.int32), tail])
        s["seq"] = torch.cat([torch.arange(b, device="cuda", dtype=torch.int32).repeat_interleave(n), tail])
        s["q_out"] = torch.zeros((rows + c["pad"], nq, d), device="cuda", dtype=wide)
        s["k_out"] = torch.zeros((rows + c["pad"], nk, d), device="cuda", dtype=wide) if c["k_out"] else None
        held = (b, nk, s["table"].shape[1] * c["ps"])
        s["position"] = torch.zeros(held, device="cuda", dtype=torch.int32) if c["track"] else None
        s["weight"] = torch.ones(held, device="cuda") if c["track"] else None
        return s
    lens = _lens(c)
    s["table"], pages = _table(c, gen, lens, max(lens))
    s["k_cache"], s["v_cache"] = _pool(c, gen, pages)
    s["lens"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
    held = (c["batch"], c["n_kv"], s["table"].shape[1] * c["ps"])
    # what rows received so far: a few heavy ones, a long tail, and rows too new to have any
    heavy = torch.randn(held, generator=gen, device="cuda").mul_(2.0).exp_()
    s["weight"] = heavy * (torch.rand(held, generator=gen, device="cuda") > 0.05)
    s["weight_out"] = torch.zeros(held, device="cuda")
    if c["op"] == "attend":
        q = torch.randn((c["batch"], c["n_q"], c["d"]), generator=gen, device="cuda", dtype=wide)
        s["q"] = q * torch.linspace(0.5, 3.0, c["n_q"], device="cuda")[None, :, None].to(wide)   # flat and peaked heads
        s["out"] = torch.zeros_like(q)
        s["lse"] = torch.zeros((c["batch"], c["n_q"]), device="cuda")
        return s
    # positions: distinct, and not in order any more once rows have been given up before
    n = held[2]
    order = torch.rand((c["batch"], c["n_kv"], n), generator=gen, device="cuda").argsort(-1).to(torch.int32)
    inside = torch.arange(n, device="cuda")[None, None] < s["lens"][:, None, None]
    s["position"] = torch.where(inside, 3 * order + 1, 0).to(torch.int32)
    s["position_out"] = torch.zeros(held, device="cuda", dtype=torch.int32)
    s["lens_out"] = torch.zeros_like(s["lens"])
    return s


# ------------------------------------------------------------------ plain forms

def _bytes(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e5m2 else x


def _rotate(x, w, cos, sin, rd):
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
    a, z = x[..., :rd // 2], x[..., rd // 2:rd]
    return torch.cat([a * cos - z * sin, z * cos + a * sin, x[..., rd:]], -1)


def _plain_norm(s):
    c = s["case"]
    rd = c["rd"]
    live = (s["positions"] >= 0).nonzero().flatten()
    pos, seq, at = s["positions"][live], s["seq"][live].long(), s["index"][live].long()
    theta = BASE ** (-2.0 * torch.arange(rd // 2, device="cuda", dtype=torch.float64) / rd)
    angle = pos.double()[:, None] * theta[None]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    q = _rotate(s["q"][live], s["q_weight"], cos, sin, rd).to(s["q"].dtype)
    k = _rotate(s["k"][live], s["k_weight"], cos, sin, rd).to(s["k"].dtype)
    s["q_out"][live] = q
    if s["k_out"] is not None:
        s["k_out"][live] = k
    page, row = s["table"][seq, at // c["ps"]].long(), at % c["ps"]
    s["k_cache"][page, :, row] = k
    _bytes(s["v_cache"])[page, :, row] = _bytes(s["v"][live].to(s["v_cache"].dtype))
    if s["position"] is not None:
        s["position"][seq, :, at] = pos[:, None].expand(-1, c["n_kv"])
        s["weight"][seq, :, at] = 0.0
    return _norm_outputs(s)


def _norm_outputs(s):
    return {n: s[n] for n in ("q_out", "k_out", "k_cache", "v_cache", "position", "weight") if s[n] is not None}


def _plain_attend(s):
    c = s["case"]
    nk, d = c["n_kv"], c["d"]
    b, width = s["table"].shape
    g, n = c["n_q"] // nk, width * c["ps"]
    page = s["table"].clamp(min=0).long()
    inside = torch.arange(n, device="cuda")[None] < s["lens"][:, None]                       # [b][n]
    k = s["k_cache"][page].permute(0, 2, 1, 3, 4).reshape(b, nk, n, d).float()
    z = torch.matmul(s["q"].float().view(b, nk, g, d), k.transpose(-1, -2)) / math.sqrt(d)
    del k
    z = z.masked_fill(~inside[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True).clamp(min=-1e30)
    z = torch.exp(z - top)
    total = z.sum(-1, keepdim=True)
    v = _bytes(s["v_cache"])[page].view(s["v_cache"].dtype).permute(0, 2, 1, 3, 4).reshape(b, nk, n, d).float()
    v = v.masked_fill(~inside[:, None, :, None], 0.0)
    z = z / torch.where(total == 0, 1.0, total)
    out = torch.matmul(z, v).reshape(b, c["n_q"], d).to(s["q"].dtype)
    lse = torch.where(total == 0, -math.inf, top + torch.log(total)).reshape(b, c["n_q"])
    if not c["weigh"]:
        return {"out": out, "lse": lse}
    added = torch.where(inside[:, None], s["weight"] + z.sum(2), s["weight_out"])
    return {"out": out, "lse": lse, "weight": added}


def _plain_evict(s):
    c = s["case"]
    ps, budget = c["ps"], c["budget"]
    n = s["weight"].shape[2]
    at = torch.arange(n, device="cuda")
    inside = at[None, None] < s["lens"][:, None, None]
    pos = s["position"]
    last = torch.where(inside, pos, -1).amax(-1, keepdim=True)
    safe = (pos > last - c["recent"]) | (pos < c["sink"])
    key = torch.where(inside, torch.where(safe, math.inf, s["weight"]), -math.inf)
    rank = key.sort(dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(inside.expand_as(key).contiguous()).scatter_(-1, rank[..., :budget], True) & inside
    hole = ~kept & inside & (at < budget)
    moved = kept & (at >= budget)
    b_to, h_to, to = hole.nonzero(as_tuple=True)
    b_of, h_of, of = moved.nonzero(as_tuple=True)
    p_to, p_of = s["table"][b_to, to // ps].long(), s["table"][b_of, of // ps].long()
    for x in (s["k_cache"], _bytes(s["v_cache"])):
        x[p_to, h_to, to % ps] = x[p_of, h_of, of % ps]
    stays = kept & (at < budget)
    for name in ("position", "weight"):
        out = s[name + "_out"]
        out.copy_(torch.where(stays, s[name], out))
        out[b_to, h_to, to] = s[name][b_of, h_of, of]
    s["lens_out"].copy_(s["lens"].clamp(max=budget))
    return _evict_outputs(s)


def _evict_outputs(s):
    return {n: s[n] for n in ("k_cache", "v_cache", "position_out", "weight_out", "lens_out")}


# ------------------------------------------------------------------ one pass

def run(s):
    c = s["case"]
    if not own:
        return {"norm": _plain_norm, "attend": _plain_attend, "evict": _plain_evict}[c["op"]](s)
    import sparse_kv_cache_gb300 as skv
    if c["op"] == "norm":
        skv.qk_norm_rope(s["q"], s["k"], s["positions"], s["q_out"], s["k_out"], q_weight=s["q_weight"],
                         k_weight=s["k_weight"], eps=EPS, rope_base=BASE, rotary_dim=c["rd"], v=s["v"],
                         k_cache=s["k_cache"], v_cache=s["v_cache"], table=s["table"], seq=s["seq"], index=s["index"],
                         position=s["position"], weight=s["weight"])
        return _norm_outputs(s)
    if c["op"] == "attend":
        weigh = dict(weight=s["weight"], weight_out=s["weight_out"]) if c["weigh"] else {}
        skv.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["out"], lse=s["lse"], **weigh)
        out = {"out": s["out"], "lse": s["lse"]}
        return {**out, "weight": s["weight_out"]} if c["weigh"] else out
    skv.paged_evict(s["k_cache"], s["v_cache"], s["table"], s["lens"], s["weight"], s["position"], budget=c["budget"],
                    recent=c["recent"], sink=c["sink"], lens_out=s["lens_out"], weight_out=s["weight_out"],
                    position_out=s["position_out"])
    return _evict_outputs(s)


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(c, seed):
    s = prepare(c, seed)
    return {"norm": _exact_norm, "attend": _exact_attend, "evict": _exact_evict}[c["op"]](s)


def _turn(x, w, pos, rd):
    """RMS norm and rotation of x [rows][heads][d] as complex numbers."""
    x = x.double()
    x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.double()
    freq = torch.exp(torch.arange(rd // 2, dtype=torch.float64, device=x.device) * (-2.0 * math.log(BASE) / rd))
    phase = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), pos.double()[:, None] * freq)
    y = torch.complex(x[..., :rd // 2].contiguous(), x[..., rd // 2:rd].contiguous()) * phase[:, None]
    return torch.cat([y.real, y.imag, x[..., rd:]], -1)


def _exact_norm(s):
    """q, k as defined; what is copied or set (values, positions, weights) has no value here."""
    c = s["case"]
    q, k = s["q_out"].double(), s["k_out"].double() if s["k_out"] is not None else None
    cache = s["k_cache"].double()
    n = c["batch"] * c["tokens"]
    for lo in range(0, n, 8192):
        hi = min(n, lo + 8192)
        pos = s["positions"][lo:hi]
        q[lo:hi] = _turn(s["q"][lo:hi], s["q_weight"], pos, c["rd"])
        rot = _turn(s["k"][lo:hi], s["k_weight"], pos, c["rd"])
        if k is not None:
            k[lo:hi] = rot
        i, at = s["seq"][lo:hi].long(), s["index"][lo:hi].long()
        cache[s["table"][i, at // c["ps"]].long(), :, at % c["ps"]] = rot
    got = {"q_out": q, "k_cache": cache, "v_cache": None}
    if k is not None:
        got["k_out"] = k
    return got


def _exact_attend(s):
    c = s["case"]
    g = c["n_q"] // c["n_kv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    weight = s["weight_out"].double()
    for i, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        pages = s["table"][i, :-(-n // c["ps"])].long()
        for h in range(c["n_kv"]):
            heads = slice(h * g, (h + 1) * g)
            k = s["k_cache"][pages, h].reshape(-1, c["d"])[:n].double()
            z = (s["q"][i, heads].double() @ k.T) * c["d"] ** -0.5
            lse[i, heads] = z.logsumexp(-1)
            p = (z - lse[i, heads, None]).exp()
            v = s["v_cache"][:, h].view(torch.uint8)[pages].view(s["v_cache"].dtype) if c["kind"] == "fp8" else s["v_cache"][pages, h]
            out[i, heads] = p @ v.reshape(-1, c["d"])[:n].double()
            weight[i, h, :n] = s["weight"][i, h, :n].double() + p.sum(0)
    return {"out": out, "lse": lse, "weight": weight} if c["weigh"] else {"out": out, "lse": lse}


def _exact_evict(s):
    """The kept weights, by a sort of each unit on the host; rows, positions and lengths are copies and counts."""
    c = s["case"]
    weight, pos = s["weight"].double().cpu().numpy(), s["position"].cpu().numpy().astype(np.int64)
    out = s["weight_out"].double().cpu().numpy()
    for i, n in enumerate(s["lens"].tolist()):
        for h in range(c["n_kv"]):
            w, p = weight[i, h, :n], pos[i, h, :n]
            if n <= c["budget"]:
                out[i, h, :n] = w
                continue
            safe = (p > p.max() - c["recent"]) | (p < c["sink"])
            best = np.lexsort((np.arange(n), -w, ~safe))[:c["budget"]]
            stay, move = np.sort(best[best < c["budget"]]), np.sort(best[best >= c["budget"]])
            out[i, h, stay] = w[stay]
            out[i, h, np.setdiff1d(np.arange(c["budget"]), stay)] = w[move]
    return {"k_cache": None, "v_cache": None, "position_out": None, "weight_out": torch.from_numpy(out), "lens_out": None}
