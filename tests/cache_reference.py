"""The paged 8-bit cache, written from its definition: codes by torch's float8 types on the CPU,
attention in float64. Nothing here is shared with the library."""
import math

import numpy as np
import torch

F8 = {0: torch.float8_e4m3fn, 1: torch.float8_e5m2}
LARGEST = {0: 448.0, 1: 57344.0}
EMAX = {0: 8, 1: 15}


def scale_byte(amax, fmt, ceil):
    """Of fp32 magnitudes [..]: the byte of the floor or the ceil rule, 255 where not finite."""
    amax = amax.double()
    mant, ex = torch.frexp(amax)                       # mant in [1/2, 1)
    e = ex - 1 - EMAX[fmt]
    if ceil:
        e = e + (mant > LARGEST[fmt] / 2.0 ** (EMAX[fmt] + 1)).int()
    # values below the least normal fp32 count as exponent -127, like zero
    e = torch.where(amax < 2.0 ** -126, torch.full_like(e, -127), e)
    b = (e + 127).clamp(0, 254)
    return torch.where(torch.isfinite(amax), b, torch.full_like(b, 255))


def to_codes(v, fmt):
    big = LARGEST[fmt]
    return v.clamp(-big, big).float().to(F8[fmt]).view(torch.uint8)


class Cache:
    """kq, vq, ks, vs and the page table, on the CPU."""

    def __init__(self, n_pages, heads, page, dim, fmt=0, seed=0, fill="random"):
        g = torch.Generator().manual_seed(seed)
        byte = lambda *s: torch.randint(0, 256, s, generator=g, dtype=torch.uint8)  # noqa: E731
        self.page, self.dim, self.heads, self.fmt = page, dim, heads, fmt
        self.kq, self.vq = byte(n_pages, heads, page, dim), byte(n_pages, heads, page // 32, dim, 32)
        self.ks, self.vs = byte(n_pages, heads, page // 32), byte(n_pages, heads, page // 32)
        self.g = g

    def tensors(self):
        return self.kq, self.ks, self.vq, self.vs

    def block(self, table, pos):
        """(page, block in it) of a position, or None."""
        p = pos // self.page
        if p >= len(table) or pos < 0:
            return None
        page = int(table[p])
        return (page, pos % self.page // 32) if 0 <= page < self.kq.shape[0] else None

    def _codes(self, x, at):
        """The block's codes [heads][32][dim], a view that can be written."""
        page, i = at
        return self.kq[page, :, 32 * i:32 * i + 32] if x == "k" else self.vq[page, :, i].transpose(1, 2)

    def write(self, k, v, table, length, ceil=False):
        """The newest len(k) tokens of a sequence, positions length - len(k) on."""
        n = k.shape[0]
        for first in range((length - n) // 32 * 32, length, 32):
            at = self.block(table, first)
            lo, hi = max(length - n - first, 0), min(length - first, 32)
            if at is None or lo >= hi:
                continue
            r = first + lo - (length - n)
            for x, t in (("k", k), ("v", v)):
                new = t[r:r + hi - lo].float().transpose(0, 1)
                amax = new.abs().amax((1, 2))
                amax = torch.where(torch.isnan(new).any(2).any(1), torch.tensor(math.inf), amax)
                s = self.ks if x == "k" else self.vs
                e = scale_byte(amax, self.fmt, ceil)
                was = s[at[0], :, at[1]].int()
                if lo > 0:
                    e = torch.maximum(e, was)
                q = self._codes(x, at)
                f = torch.exp2((127 - e).double())[:, None, None]
                code = to_codes(torch.nan_to_num(new.double(), 0, 0, 0) * f, self.fmt)
                code[e == 255] = 0
                if lo > 0:
                    held = q[:, :lo].contiguous().view(F8[self.fmt]).double()
                    again = to_codes(held * torch.exp2((was - e).double())[:, None, None], self.fmt)
                    again[e == 255] = 0
                    q[:, :lo] = torch.where((e > was)[:, None, None], again, q[:, :lo])
                q[:, lo:hi] = code
                s[at[0], :, at[1]] = e.to(torch.uint8)

    def tokens(self, x, table, first, count):
        """Tokens in float64 [count][heads][dim] and which of them exist."""
        out = torch.zeros((count, self.heads, self.dim), dtype=torch.float64)
        has = torch.zeros(count, dtype=torch.bool)
        for i in range(count):
            at = self.block(table, first + i)
            if at is None:
                continue
            has[i] = True
            q = self._codes(x, at)[:, (first + i) % 32].contiguous().view(F8[self.fmt]).double()
            s = (self.ks if x == "k" else self.vs)[at[0], :, at[1]]
            f = torch.exp2(s.double() - 127)
            f[s == 255] = math.nan
            out[i] = q * f[:, None]
        return out, has

    def random_sequence(self, table, length, seed, spread=1.0):
        """Writes `length` random tokens and returns nothing: slots behind them keep their bytes."""
        g = torch.Generator().manual_seed(seed)
        kv = torch.randn((2, length, self.heads, self.dim), generator=g)
        kv = kv * torch.exp(spread * torch.randn((2, length, self.heads, 1), generator=g))
        self.write(kv[0], kv[1], table, length)


def attention(cache, q, table, length, scale, p_eps):
    """Rows [n][query heads][dim] of a sequence's newest tokens -> (out, lse, tolerance without the
    output's rounding), all float64. The tolerance, with u = 2^-24: a score's fp32 sum of dim exact
    products drops and rounds at most dim + 8 units of sum |q k|, which is its probability's relative
    error; the scaling to the base of two, the subtraction of the maximum and the exponential add 8
    units of the largest |score| and 8 of one. Each enters the numerator and the denominator. The
    probabilities' rounding p_eps enters the numerator only. Sums over tokens: one rounding for 8 of
    them at most, 64 for the joints, 3 terms a product."""
    n, heads, dim = q.shape
    u = 2.0 ** -24
    k, has = cache.tokens("k", table, 0, length)
    v, _ = cache.tokens("v", table, 0, length)
    group = heads // cache.heads
    out = torch.zeros((n, heads, dim), dtype=torch.float64)
    tol = torch.zeros_like(out)
    lse = torch.full((n, heads), -math.inf, dtype=torch.float64)
    for t in range(n):
        seen = length - n + t + 1
        keep = has[:seen] if seen > 0 else has[:0]
        if not keep.any():
            continue
        kk, vv = k[:seen][keep], v[:seen][keep]
        for h in range(heads):
            x = q[t, h].double()
            kh, vh = kk[:, h // group], vv[:, h // group]
            s = kh @ x * scale
            size = (kh.abs() @ x.abs() * abs(scale)).max()
            w = torch.softmax(s, 0)
            # a NaN value makes the row NaN even where its weight is zero
            out[t, h] = w @ vh
            lse[t, h] = torch.logsumexp(s, 0)
            rel = (dim + 8) * u * size + 8 * u * s.abs().max() + 8 * u
            tol[t, h] = (2 * rel + p_eps + (3 * seen / 8 + 64) * u) * (w @ vh.abs())
    return out, lse, tol


def table_of(lengths, page, spare=1, seed=0, width=None):
    """A page table [B][width] int32 of distinct pages in any order and the number of pages."""
    need = [-(-max(n, 0) // page) for n in lengths]
    rng = np.random.default_rng(seed)
    order = rng.permutation(sum(need) + spare)
    width = width or max(need + [1])
    t = np.full((len(lengths), width), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = order[at:at + n]
        at += n
    return torch.from_numpy(t), sum(need) + spare
