"""Plain 64-bit references of the paged attention operators, and seeded cases.

Everything here runs on the CPU in numpy, from the definitions alone: the block
tables and slot maps request by request, the attention row by row over every
position of the request.  Caches are filled with NaN wherever no visible key
lies, so that anything read by mistake shows.
"""
from __future__ import annotations

import math
from dataclasses import dataclass

import numpy as np
import torch

# half a step of each type, relative to the value
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


@dataclass
class Case:
    q: torch.Tensor
    k_cache: torch.Tensor
    v_cache: torch.Tensor
    table: torch.Tensor
    cu: torch.Tensor
    seq: torch.Tensor
    keys: list          # per request [seq, Hkv, D] K and V rows as stored
    values: list


def make(ctx, new, hq, hkv, dim, page, dtype, seed=0, pad_rows=0, extra_cols=2, scale_k=1.0,
         holes=()):
    """ctx / new: cached and new tokens per request.  holes: (request, page index)
    table entries without a page (their positions hold no key)."""
    g = torch.Generator().manual_seed(seed)
    n = len(ctx)
    total = [c + t for c, t in zip(ctx, new)]
    used = [-(-t // page) for t in total]
    num_pages = sum(used) + 2
    ids = torch.randperm(num_pages, generator=g)
    cols = max(used + [0]) + extra_cols
    table = torch.full((n, cols), -1, dtype=torch.int32)
    kc = torch.full((num_pages, hkv, page, dim), float("nan"), dtype=dtype)
    vc = torch.full((num_pages, hkv, page, dim), float("nan"), dtype=dtype)
    keys, values, at = [], [], 0
    for i in range(n):
        table[i, :used[i]] = ids[at:at + used[i]].to(torch.int32)
        at += used[i]
        k = (scale_k * torch.randn(total[i], hkv, dim, generator=g)).to(dtype)
        v = torch.randn(total[i], hkv, dim, generator=g).to(dtype)
        j = torch.arange(total[i])
        pg = table[i, j // page].long()
        kc[pg, :, j % page] = k
        vc[pg, :, j % page] = v
        keys.append(k)
        values.append(v)
    for i, p in holes:
        table[i, p] = -1
    cu = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32)
    q = torch.randn(int(cu[-1]) + pad_rows, hq, dim, generator=g).to(dtype)
    return Case(q, kc, vc, table, cu, torch.tensor(total, dtype=torch.int32), keys, values)


def attention(c, page, scale, window=0, sinks=0, rows=None):
    """(out, lse, tol_out, tol_lse) in 64 bits, of all rows or of the listed ones.  The tolerances follow the rounding
    steps of an fp32 softmax: a score is a dot product of D terms, its exponent
    a difference of numbers up to X; every weight is off by at most the relative
    w below, the probabilities are rounded to the input type (half a step each)
    before the product with V, and out once more."""
    dtype = c.q.dtype
    half = HALF[dtype]
    T, hq, dim = c.q.shape
    hkv = c.k_cache.shape[1]
    group = hq // hkv
    out, lse = np.zeros((T, hq, dim)), np.full((T, hq), -np.inf)
    tol, tol_lse = np.zeros((T, hq, dim)), np.zeros((T, hq))
    q = c.q.double().numpy()
    for i in range(len(c.keys)):
        a, b = int(c.cu[i]), int(c.cu[i + 1])
        L = int(c.seq[i])
        k, v = c.keys[i].double().numpy(), c.values[i].double().numpy()
        j = np.arange(L)
        paged = np.array([x // page < c.table.shape[1] and int(c.table[i, x // page]) >= 0
                          for x in range(L)], dtype=bool)
        for x in range(a, b):
            if rows is not None and x not in rows:
                continue
            p = L - (b - a) + (x - a)
            see = (j <= p) & paged
            if window:
                see &= (p - j < window) | (j < sinks)
            idx = np.nonzero(see)[0]
            if idx.size == 0:
                continue
            for h in range(hq):
                kk, vv = k[idx, h // group], v[idx, h // group]
                with np.errstate(all="ignore"):
                    s = scale * (kk @ q[x, h])
                    top = s.max()
                    e = np.exp(s - top)
                    w = e / e.sum()
                    out[x, h] = w @ vv
                    lse[x, h] = top + math.log(e.sum())
                    dots = abs(scale) * (np.abs(kk) @ np.abs(q[x, h])).max()
                    rel = 2.0 ** -24 * (2 * (dim + 4) * dots + 6 * np.abs(s).max() + idx.size + 16)
                    A = w @ np.abs(vv)
                p_round = 0.0 if dtype == torch.float32 else half
                # fp16 leaves its normal range below 2^-14: the probabilities (scaled by 2^6)
                # and the output are then off by half of its smallest step, 2^-25
                most = np.abs(vv[np.isfinite(vv)]).max(initial=0.0)
                tiny = idx.size * 2.0 ** -31 * most + 2.0 ** -25 if dtype == torch.float16 else 0.0
                tol[x, h] = A * (p_round + 2 * rel) + half * np.abs(out[x, h]) + tiny
                tol_lse[x, h] = 2 * rel + 2.0 ** -22 * (abs(lse[x, h]) + 1)
    return out, lse, tol, tol_lse


def tables(ctx, new, free, table, page, num_pages, max_tokens):
    """The step's tables by the definition, in plain Python."""
    table = table.clone()
    cu, seq, slots, pos, taken = [0], [], [], [], 0
    for i, (c, t) in enumerate(zip(ctx, new)):
        c, t = max(c, 0), max(t, 0)
        have, want = -(-c // page), -(-(c + t) // page)
        fresh = {}
        for p in range(have, want):
            pid = int(free[taken]) if taken < len(free) else -1
            fresh[p] = pid
            if p < table.shape[1]:
                table[i, p] = pid
            taken += 1
        for x in range(c, c + t):
            p = x // page
            pid = int(table[i, p]) if p < table.shape[1] else -1
            slots.append(pid * page + x % page if 0 <= pid < num_pages else -1)
            pos.append(x)
        cu.append(cu[-1] + t)
        seq.append(c + t)
    pad = max_tokens - len(slots)
    return (torch.tensor(cu, dtype=torch.int32), torch.tensor(seq, dtype=torch.int32),
            torch.tensor(slots + [-1] * pad, dtype=torch.int64),
            torch.tensor(pos + [-1] * pad, dtype=torch.int32),
            torch.tensor([taken], dtype=torch.int32), table)
