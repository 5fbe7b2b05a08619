"""Inputs and comparisons of the paged-cache tests (no arithmetic of the operators)."""
import numpy as np
import torch

KINDS = {"bf16": (torch.bfloat16, torch.bfloat16), "f32": (torch.float32, torch.float32),
         "fp8": (torch.bfloat16, torch.float8_e5m2)}


def f64(t):
    """A tensor's exact values in float64 numpy."""
    return t.detach().cpu().to(torch.float32).double().numpy()


class Paged:
    """A paged cache of random rows.  Whatever no row uses -- the rest of last pages, spare pages --
    is NaN, and table entries without a page are -1, so that reading them shows."""

    def __init__(self, kind, lens, heads, d, ps, layout="hnd", seed=0, cap=None, spare=2, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.kind, self.heads, self.d, self.ps = kind, heads, d, ps
        self.n = list(lens)
        need = [-(-n // ps) for n in self.n]
        width = max(max(need, default=1), 1, -(-(cap or 0) // ps))
        pages = sum(-(-max(n, cap or 0) // ps) for n in self.n) + spare
        ids = torch.randperm(pages, generator=g)
        table = torch.full((len(self.n), width), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(self.n):
            own = -(-max(n, cap or 0) // ps)
            table[b, :own] = ids[at:at + own].to(torch.int32)
            at += own
        wide, val = KINDS[kind]
        # rows as the cache stores them, [sequence][head][row][d]
        self.krows = [torch.randn((heads, n, d), generator=g).to(wide) for n in self.n]
        self.vrows = [torch.randn((heads, n, d), generator=g).to(val) for n in self.n]
        shape = (pages, heads, ps, d) if layout == "hnd" else (pages, ps, heads, d)
        k = torch.full(shape, float("nan")).to(wide)
        v = torch.full(shape, float("nan")).to(val)
        if layout != "hnd":
            k, v = k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)
        for b, n in enumerate(self.n):
            for p in range(need[b]):
                lo, hi = p * ps, min(n, (p + 1) * ps)
                k[int(table[b, p]), :, :hi - lo] = self.krows[b][:, lo:hi]
                v.view(torch.uint8 if kind == "fp8" else val)[int(table[b, p]), :, :hi - lo] = \
                    self.vrows[b][:, lo:hi].view(torch.uint8 if kind == "fp8" else val)
        self.k, self.v, self.table = k.to(device), v.to(device), table.to(device)
        self.lens = torch.tensor(self.n, dtype=torch.int32, device=device)
        self.rows = width * ps

    def stored(self, which, b, h, n):
        """The first n rows of a unit as the pools hold them now, float64."""
        pool = self.k if which == "k" else self.v
        t = self.table[b].cpu()
        out = np.empty((n, self.d))
        host = pool[:, h].cpu().float() if pool.dtype != torch.float8_e5m2 else pool[:, h].cpu().to(torch.float32)
        for i in range(n):
            out[i] = host[int(t[i // self.ps]), i % self.ps].double().numpy()
        return out
