"""A paged cache with known contents, and the attention over it in 64 bits.

Independent of the library: caches are filled by plain indexing, e4m3 codes and
exponents by the definition in include/sv_attention.h with torch's own
conversion, and every query is computed from the slice of keys that it sees, so
that nothing outside the slice can reach it.
"""
import math

import torch

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def quantise(x):
    """(codes uint8, exponent bytes uint8) of the vectors along the last axis."""
    f = x.double()
    if x.dtype == torch.float16:
        f = torch.where(f.isfinite(), f.clamp(-61440.0, 61440.0), f)
    top = f.abs().amax(-1)
    bad = ~f.isfinite().all(-1)
    mantissa, e = torch.frexp(torch.where(bad, 1.0, top))
    e = torch.where(mantissa <= 0.875, e - 9, e - 8)
    e = torch.where(top > 0, e.clamp(min=-117), torch.full_like(e, -117))
    y = torch.ldexp(f, -e.unsqueeze(-1)).float()  # exact: a float's exponent moved
    y = torch.where(bad.unsqueeze(-1), 0.0, y)
    code = y.to(torch.float8_e4m3fn).view(torch.uint8)
    return code, torch.where(bad, 255, e + 127).to(torch.uint8)


def values(code, exp):
    """The numbers that codes and exponent bytes stand for, in 64 bits."""
    e = torch.where(exp == 255, math.nan, exp.double() - 127.0)
    return code.view(torch.float8_e4m3fn).double() * torch.exp2(e).unsqueeze(-1)


class Cache:
    """Pages of a random order, every slot set. `keys`, `values`: what sequence b's positions
    hold, in 64 bits, [positions, heads, d]."""

    def __init__(self, lens, chunks, heads, d, page, dtype="bf16", e4m3=False, heads_first=False,
                 seed=0, spread=1.0, spare=3, fill=None, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.chunks, self.page, self.e4m3 = list(lens), list(chunks), page, e4m3
        self.heads, self.d, self.dtype = heads, d, DTYPES[dtype]
        B = len(self.lens)
        need = [-(-(n + t) // page) for n, t in zip(self.lens, self.chunks)]
        pool = sum(need) + spare
        order = torch.randperm(pool, generator=g).tolist()
        table = torch.full((B, max(need + [1]) + 1), -1, dtype=torch.int32)
        shape = (pool, heads, page, d) if heads_first else (pool, page, heads, d)
        self.parts = []
        for _ in range(2):
            x = (torch.randn(shape, generator=g) * spread).to(self.dtype).to(device)
            if heads_first:
                x = x.transpose(1, 2)
            self.parts.append(x)
        at = 0
        self.pages_of = []
        for b in range(B):
            mine = order[at:at + need[b]]
            at += need[b]
            table[b, :need[b]] = torch.tensor(mine, dtype=torch.int32)
            self.pages_of.append(mine)
        self.unused = order[at:]
        # What no position holds: the spare pages and the last pages' ends.
        if fill is not None:
            for x in self.parts:
                x[self.unused] = fill
                for b in range(B):
                    n = self.lens[b] + self.chunks[b]
                    if need[b] and n % page:
                        x[self.pages_of[b][-1], n % page:] = fill
        self.exps = [None, None]
        if e4m3:
            for i, x in enumerate(self.parts):
                code, e = quantise(x)
                self.parts[i] = code.view(torch.float8_e4m3fn)
                self.exps[i] = e
        self.table = table.to(device)
        self.cached = torch.tensor(self.lens, dtype=torch.int32, device=device)
        starts = torch.zeros(B + 1, dtype=torch.int32)
        starts[1:] = torch.cumsum(torch.tensor(self.chunks, dtype=torch.int64), 0)
        self.starts = starts.to(device)
        self.tokens = int(starts[-1])

    def args(self):
        return (self.parts[0], self.parts[1], self.table, self.cached, self.starts)

    def exp_args(self):
        return dict(k_exps=self.exps[0], v_exps=self.exps[1])

    def dense(self, i, b, n):
        """Positions 0 .. n - 1 of sequence b's keys (i = 0) or values (1), in 64 bits."""
        p = torch.arange(n, device=self.table.device)
        page, slot = self.table[b].long()[p // self.page], p % self.page
        if self.e4m3:
            return values(self.parts[i].view(torch.uint8)[page, slot], self.exps[i][page, slot])
        return self.parts[i][page, slot].double()


def reference(cache, query, scale, window=0):
    """out, lse and the bound on each output's error, from the definition in 64 bits.

    The bound, with u half a step of the output's type, n keys, d the head size, A = sum p |v|:
      u |out|            the output's rounding
      u A                the weights' rounding before the second product
      2 ds A             a score's error ds = (d + 8) 2^-24 scale max sum|q k| + 2^-22 |s| moves a
                         weight by ds and the normaliser by ds at most
      (n + d) 2^-23 A    sums of n terms in float32, of weights and of products
      2^-20 A            the exponentials (2^-22 each) and the division
      2^-24 sum |v|      float16 weights below 2^-14 of the row's reference
    """
    N, Hq, d = query.shape
    G = Hq // cache.heads
    out = torch.full((N, Hq, d), math.nan, dtype=torch.float64, device=query.device)
    tol = torch.zeros_like(out)
    lse = torch.full((N, Hq), math.nan, dtype=torch.float64, device=query.device)
    tol_lse = torch.zeros_like(lse)
    u = half_step(query.dtype)
    r = 0
    for b in range(len(cache.lens)):
        total = cache.lens[b] + cache.chunks[b]
        k, v = cache.dense(0, b, total), cache.dense(1, b, total)
        for t in range(cache.chunks[b]):
            p = cache.lens[b] + t
            lo = max(0, p - window + 1) if window else 0
            kk = k[lo:p + 1].repeat_interleave(G, 1)  # [n, Hq, d]
            vv = v[lo:p + 1].repeat_interleave(G, 1)
            q = query[r].double()
            prod = kk * q
            s = prod.sum(-1) * scale  # [n, Hq]
            z = torch.logsumexp(s, 0)
            w = torch.exp(s - z)
            o = (w.unsqueeze(-1) * vv).sum(0)
            a = (w.unsqueeze(-1) * vv.abs()).sum(0)
            n = p + 1 - lo
            ds = (d + 8) * 2.0 ** -24 * abs(scale) * prod.abs().sum(-1).amax(0) \
                + 2.0 ** -22 * s.abs().amax(0)
            out[r], lse[r] = o, z
            tol[r] = u * o.abs() + (u + 2 * ds.unsqueeze(-1) + (n + d) * 2.0 ** -23
                                    + 2.0 ** -20) * a + 2.0 ** -24 * vv.abs().sum(0)
            tol_lse[r] = ds + n * 2.0 ** -24 + 2.0 ** -22 * (1 + z.abs())
            r += 1
    return out, lse, tol, tol_lse


def check(out, lse, cache, query, scale, window=0, rows=None):
    ref, z, tol, tol_z = reference(cache, query, scale, window)
    rows = slice(None) if rows is None else rows
    got = out.double()[rows]
    ref, tol = ref[rows], tol[rows]
    fine = ref.isfinite()
    assert torch.equal(fine, got.isfinite()), "finite outputs differ"
    err = (got - ref).abs()
    over = (err > tol) & fine
    assert not over.any(), f"{int(over.sum())} outputs off: worst {float((err / tol)[over].max()):.3g} x"
    if lse is not None:
        fine = z[rows].isfinite()
        err = (lse.double()[rows] - z[rows]).abs()
        assert torch.equal(fine, lse[rows].isfinite())
        over = (err > tol_z[rows]) & fine
        assert not over.any(), f"lse: worst {float((err / tol_z[rows])[over].max()):.3g} x"
