"""Plain 64-bit references of the paged cache in 8 bits, and seeded cases.

Codes are bytes here and everything runs on the CPU in numpy, from the definitions alone: e4m3 from
the list of its numbers, scales by trying powers of two, an append block by block.
"""
from __future__ import annotations

import math

import numpy as np
import torch

import paged_ref as R

DTYPE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
MOST = {"e4m3": 448.0, "int8": 127.0}
UNUSED = {"e4m3": 0x7f, "int8": 0x80}       # NaN, and the code that nothing is rounded to


def _e4m3(c):
    e, m = (c >> 3) & 15, c & 7
    if c & 127 == 127:
        return math.nan
    x = math.ldexp(8 + m, e - 10) if e else math.ldexp(m, -9)
    return -x if c & 128 else x


VALUES = {"e4m3": np.array([_e4m3(c) for c in range(256)]),
          "int8": np.arange(256, dtype=np.uint8).view(np.int8).astype(np.float64)}


def nearest(y, code):
    """The codes of fp64 values within the codes' range: nearest, ties to the even code."""
    y = np.asarray(y, dtype=np.float64)
    if code == "int8":
        z = np.clip(np.where(np.isnan(y), 0.0, y), -127, 127)
        return np.rint(z).astype(np.int8).view(np.uint8)
    grid = VALUES["e4m3"][:127]
    mag = np.where(np.isfinite(y), np.abs(y), 0.0)
    hi = np.clip(np.searchsorted(grid, mag), 1, 126)
    lo = hi - 1
    a, b = mag - grid[lo], grid[hi] - mag
    c = np.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)
    c = np.where(np.isfinite(y), c, 127)
    return (c + 128 * np.signbit(y)).astype(np.uint8)


def least_scale(top, code):
    e = -126
    while math.ldexp(MOST[code], e) < top:
        e += 1
    return math.ldexp(1.0, e)


class Cache:
    """K and V codes [pages, hkv, page, dim] and scales [pages, hkv, page / block]."""

    def __init__(self, pages, hkv, page, dim, block, code, scale=math.nan):
        self.code, self.page, self.block = code, page, block
        self.codes = [np.full((pages, hkv, page, dim), UNUSED[code], dtype=np.uint8) for _ in range(2)]
        self.scales = [np.full((pages, hkv, page // block), scale, dtype=np.float32) for _ in range(2)]

    def append(self, k, v, table, cu, seq):
        """Rows [T, hkv, dim] (tensors) of each request's newest positions."""
        B, P = self.block, self.page
        for x, codes, scales in zip((k, v), self.codes, self.scales):
            x = x.double().numpy()
            for i in range(len(seq)):
                rows = range(int(cu[i]), int(cu[i + 1]))
                at = {}                                 # (block) -> [(position, row)]
                for r in rows:
                    p = int(seq[i]) - len(rows) + (r - rows[0])
                    if p >= 0 and p // P < table.shape[1]:
                        at.setdefault(p // B, []).append((p, r))
                for b, new in at.items():
                    pg, off = int(table[i, b * B // P]), b * B % P
                    if not 0 <= pg < codes.shape[0]:
                        continue
                    first = new[0][0] - b * B
                    for h in range(codes.shape[1]):
                        y = np.stack([x[r, h] for _, r in new])
                        top = np.abs(y[np.isfinite(y)]).max(initial=0.0)
                        old, s = float(scales[pg, h, off // B]), least_scale(top, self.code)
                        if first > 0:
                            s = max(s, old)
                            if s > old:
                                held = codes[pg, h, off:off + first]
                                with np.errstate(invalid="ignore"):
                                    held[:] = nearest(VALUES[self.code][held] * (old / s), self.code)
                        with np.errstate(invalid="ignore"):
                            codes[pg, h, off + first:off + first + len(new)] = nearest(y / s, self.code)
                        scales[pg, h, off // B] = s

    def row(self, side, pg, off):
        """The values [hkv, dim] of one position."""
        return VALUES[self.code][self.codes[side][pg, :, off]] * \
            self.scales[side][pg, :, off // self.block].astype(np.float64)[:, None]

    def tensors(self, dev="cpu"):
        """(k_cache, v_cache, k_scale, v_scale) as the operators take them."""
        codes = [torch.from_numpy(c.copy()).to(dev).view(DTYPE[self.code]) for c in self.codes]
        return (*codes, *[torch.from_numpy(s.copy()).to(dev) for s in self.scales])

    def same(self, got):
        """Whether operator tensors hold these bytes (e4m3 has two NaN codes) and scales."""
        for c, t in zip(self.codes, got[:2]):
            b = t.cpu().view(torch.uint8).numpy()
            x, y = VALUES[self.code][c], VALUES[self.code][b]
            if not np.array_equal(np.where(np.isnan(x), 127, c), np.where(np.isnan(y), 127, b)):
                return False
        return all(np.array_equal(s.view(np.uint32), t.cpu().numpy().view(np.uint32)) or
                   np.array_equal(s, t.cpu().numpy(), equal_nan=True)
                   for s, t in zip(self.scales, got[2:]))


def make(ctx, new, hq, hkv, dim, page, block, dtype, code, seed=0, pad_rows=0, extra_cols=2, holes=()):
    """(paged_ref.Case with the values that the cache stands for, Cache).  Blocks differ in
    size; unused codes are NaN (or -128) and unused scales NaN."""
    g = torch.Generator().manual_seed(seed)
    total = [c + t for c, t in zip(ctx, new)]
    used = [-(-t // page) for t in total]
    num_pages = sum(used) + 2
    ids = torch.randperm(num_pages, generator=g)
    table = torch.full((len(ctx), max(used + [0]) + extra_cols), -1, dtype=torch.int32)
    at = 0
    for i, u in enumerate(used):
        table[i, :u] = ids[at:at + u].to(torch.int32)
        at += u
    cache = Cache(num_pages, hkv, page, dim, block, code)
    T = sum(total)
    k, v = (torch.randn(T, hkv, dim, generator=g) * torch.exp(0.4 * torch.randn(T, hkv, 1, generator=g))
            for _ in range(2))
    cache.append(k, v, table, np.cumsum([0] + total), total)
    keys, values = [], []
    for i, t in enumerate(total):
        for side, rows in ((0, keys), (1, values)):
            r = [cache.row(side, int(table[i, p // page]), p % page) for p in range(t)]
            rows.append(torch.from_numpy(np.stack(r)) if r else torch.zeros(0, hkv, dim, dtype=torch.float64))
    for i, p in holes:
        table[i, p] = -1
    cu = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32)
    q = torch.randn(int(cu[-1]) + pad_rows, hq, dim, generator=g).to(dtype)
    codes = torch.from_numpy(cache.codes[0])
    return R.Case(q, codes, codes, table, cu, torch.tensor(total, dtype=torch.int32), keys, values), cache
