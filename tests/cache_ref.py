"""Plain 64-bit reference of the paged cache's operators (CPU, torch.float64), and the tolerances that the
kernels' arithmetic allows."""
from __future__ import annotations

import math

import torch

U = 2.0 ** -8   # largest relative error of a rounding to bf16
F = 2.0 ** -24  # and to float32


def rotate(x, pos, base=10000.0, scale=1.0):
    """x [T, H, D] rotated to positions pos [T]: pairs (j, j + D/2), angle pos·scale·base^(-2j/D)."""
    x = x.double()
    half = x.shape[-1] // 2
    a = pos.double()[:, None] * scale * base ** (-torch.arange(half, dtype=torch.float64) / half)
    c, s = a.cos()[:, None], a.sin()[:, None]
    lo, hi = x[..., :half], x[..., half:]
    return torch.cat([lo * c - hi * s, hi * c + lo * s], -1)


def pack(x):
    """4-bit rows of x [.., D] (bf16 values): codes [.., D] (whole numbers), scale and min [..]."""
    x = x.double()
    mn, mx = x.min(-1).values, x.max(-1).values
    s = ((mx - mn) / 15).to(torch.bfloat16).double()
    c = torch.where(s[..., None] > 0, ((x - mn[..., None]) / s[..., None]).round().clamp(0, 15), 0.0)
    return torch.nan_to_num(c), s, mn


def split_codes(b):
    """Codes [.., D] of the stored bytes [.., D/2]."""
    b = b.to(torch.int64)
    return torch.cat([b % 16, b // 16], -1).double()


def join_codes(c):
    """Stored bytes of whole-number codes."""
    c = c.to(torch.uint8)
    half = c.shape[-1] // 2
    return c[..., :half] | (c[..., half:] << 4)


class Paged:
    """A cache built on the host from rows of each sequence: places in shuffled pages, with unused rows and table
    entries filled with what must never be used."""

    def __init__(self, lens, heads, dim, page_size, bits, seed=0, fill=float("nan"), spare=2):
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // page_size) for n in lens]
        pages = sum(need) + spare
        self.lens, self.S, self.bits, self.dim, self.heads = list(lens), page_size, bits, dim, heads
        perm = torch.randperm(pages, generator=g)
        self.table = torch.full((len(lens), max(need + [1]) + 1), -7, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n].to(torch.int32)
            at += n
        shape = (pages, heads, page_size)
        self.k, self.v = (torch.randn(*shape, dim, generator=g).bfloat16() for _ in range(2))
        self.k *= 1 + 2 * (torch.rand(1, heads, 1, dim, generator=g) < 0.05).bfloat16()
        used = torch.zeros(shape, dtype=torch.bool)
        for b, n in enumerate(lens):
            for p in range(need[b]):
                used[int(self.table[b, p]), :, : min(page_size, n - p * page_size)] = True
        self.ks = self.vs = None
        if bits == 4:
            (ck, sk, mk), (cv, sv, mv) = pack(self.k), pack(self.v)
            self.k, self.v = join_codes(ck), join_codes(cv)
            self.ks, self.vs = torch.stack([sk, mk], -1).bfloat16(), torch.stack([sv, mv], -1).bfloat16()
            for t in (self.ks, self.vs):
                t[~used] = fill
        else:
            for t in (self.k, self.v):
                t[~used] = fill

    def rows(self, b, h):
        """Keys, values [len, D] of sequence b's head h in 64 bits, and the size of what a value row's weight is
        multiplied with (the row, or scale·|code - 8|)."""
        n = self.lens[b]
        pages = self.table[b, : -(-n // self.S)].long()
        take = lambda t: t[pages, h].reshape(len(pages) * self.S, -1)[:n]  # noqa: E731
        if self.bits == 16:
            k, v = take(self.k).double(), take(self.v).double()
            return k, v, k.abs(), v.abs()
        ck, cv = split_codes(take(self.k)), split_codes(take(self.v))
        ks, vs = take(self.ks).double(), take(self.vs).double()
        k, v = ks[:, 1:] + ks[:, :1] * ck, vs[:, 1:] + vs[:, :1] * cv
        return (k, v, ks[:, :1].abs() * (128 + ck) + (ks[:, 1:] - 128 * ks[:, :1]).abs(),
                vs[:, :1].abs() * (cv - 8).abs())


def attention(cache, q, starts):
    """o [T, H, D], lse [T, H] in 64 bits of the new tokens q [T, H, D] (starts: packed starts of the new tokens), and
    the errors that the kernels may make of each.

    Scores: products of bf16 values are exact in 32 bits; a sum of D of them and the scaling are off by at most (D + 8)
    roundings of the terms' absolute sum.  The terms of 4-bit rows are q·scale·(128 + code) and q·(min - 128 scale): bf16
    holds 128 + code as it is, and the two sums are taken one from the other.  Weights: twice that, relatively, and
    2^-21 of the exponential.  o: each weight is rounded to bf16 before the product, and from bf16 rows the sum of the
    rounded ones may be what divides (2 U of a term; from 4 bits U), the sums over n keys are off by n F, and the
    result is rounded once to bf16.  lse: the scores' error, the sum's, and a few roundings of itself."""
    T, H, D = q.shape
    g = H // cache.heads
    o, lse = torch.zeros(T, H, D, dtype=torch.float64), torch.full((T, H), -math.inf, dtype=torch.float64)
    to, tl = torch.zeros_like(o), torch.zeros_like(lse)
    for b, n in enumerate(cache.lens):
        t0, t1 = int(starts[b]), int(starts[b + 1])
        if t1 == t0:
            continue
        place = n - (t1 - t0) + torch.arange(t1 - t0)
        for h in range(cache.heads):
            if n == 0:
                continue
            k, v, ka, va = cache.rows(b, h)
            for y in range(h * g, (h + 1) * g):
                x = q[t0:t1, y].double()
                z = x @ k.T / math.sqrt(D)
                za = x.abs() @ ka.T / math.sqrt(D)
                seen = torch.arange(n)[None] <= place[:, None]
                z = z.masked_fill(~seen, -math.inf)
                some = place >= 0
                zs, seen_s = z[some], seen[some]
                if not len(zs):
                    continue
                lse[t0:t1, y][some] = torch.logsumexp(zs, -1)
                p = torch.softmax(zs, -1)
                ds = ((D + 8) * F * za[some]).masked_fill(~seen_s, 0.0).amax(-1)
                rel = 2 * ds + 2.0 ** -21 + n * F
                out, size = p @ v, p @ va
                rows = torch.arange(t0, t1)[some]
                o[rows, y] = out
                to[rows, y] = U * out.abs() + ((2 * U if cache.bits == 16 else U) + rel[:, None]) * (1 + U) * size + rel[:, None] * (p @ v.abs())
                tl[rows, y] = ds + 2.0 ** -21 + n * F + 4 * F * lse[rows, y].abs()
    return o, lse, to, tl
