"""The paged cache in 8 bits on the GPU against plain 64-bit references (tests/q8_ref.py; the
attention's tolerances are those that tests/paged_ref.py derives: the values of the cache are bf16
and, in these cases, fp16 numbers, so only the probabilities and the output are rounded)."""
import numpy as np
import pytest
import torch

import paged_ref as R
import q8_ref as Q
from gated_delta_rule_65_amd import paged, paged_q8 as P8, positions
from test_paged_gpu import CASES, check

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
CODES = ["e4m3", "int8"]


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).to(DEV)


# --------------------------------------------------------------- append, read

# page, block, hkv, dim
LAYOUTS = [(16, 16, 2, 128), (16, 4, 3, 64), (48, 24, 1, 64), (20, 5, 2, 128), (64, 64, 2, 64),
           (8, 1, 2, 128), (100, 100, 1, 128), (1, 1, 2, 64), (512, 256, 1, 64)]


@pytest.mark.parametrize("dt", [BF, HF, FP])
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
def test_appends_match_the_definition(layout, code, dt):
    """Steps of ragged lengths, small rows first so that scales grow, some positions written again:
    every code and scale after each step, those that no step touches among them, and what is read back."""
    page, block, hkv, dim = layout
    g = torch.Generator().manual_seed(page * 7 + block)
    n, cols = 4, max(3, -(-130 // page))
    pages = n * cols + 3
    table = torch.randperm(pages, generator=g)[:n * cols].view(n, cols).to(torch.int32)
    cache = Q.Cache(pages, hkv, page, dim, block, code)
    dev = cache.tensors(DEV)
    seq = [0] * n
    for step in range(6):
        back = [min(s, int(torch.randint(0, 4, (1,), generator=g))) if step % 2 else 0 for s in seq]
        new = [int(torch.randint(0, 40 if step < 2 else 3, (1,), generator=g)) for _ in range(n)]
        new = [min(t, cols * page - s + b) for t, s, b in zip(new, seq, back)]
        seq = [s - b + t for s, b, t in zip(seq, back, new)]
        T = sum(new) + 2                                       # a padded batch
        size = 10.0 ** torch.randint(-3, 1 + step // 2, (T, 1, 1), generator=g)
        k, v = ((torch.randn(T, hkv, dim, generator=g) * size).to(dt) for _ in range(2))
        cu = [0] + list(np.cumsum(new))
        print("append", layout, code, dt, step, new, flush=True)
        P8.kv_append_q8(k.to(DEV), v.to(DEV), *dev, table.to(DEV), i32(cu), i32(seq))
        torch.cuda.synchronize()
        cache.append(k, v, table, cu, seq)
        assert cache.same(dev), step
    total = sum(seq)
    for out_dt in (BF, HF, FP):
        k_out, v_out = (torch.full((total + 1, hkv, dim), 9, dtype=out_dt, device=DEV) for _ in range(2))
        P8.kv_read_q8(*dev, table.to(DEV), i32([0] + list(np.cumsum(seq))), i32(seq), k_out=k_out, v_out=v_out)
        torch.cuda.synchronize()
        for side, got in ((0, k_out), (1, v_out)):
            want = np.concatenate([np.stack([cache.row(side, int(table[i, p // page]), p % page)
                                             for p in range(s)]) for i, s in enumerate(seq) if s])
            assert torch.equal(got[:total].cpu(), torch.from_numpy(want).to(out_dt))
            assert torch.all(got[total:] == 9)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dt", [BF, FP])
def test_magnitudes_at_the_scales_edges(code, dt):
    """Largest codes, ties, the least scale, zeros, the largest magnitudes, NaN and infinities."""
    most = Q.MOST[code]
    tops = [most, most * 1.0625, most * 2.0 ** 20, most * 2.0 ** -30, 2.0 ** -140, 0.0, 1.0, 2.0 ** 126, 3.0e-38,
            448.0, 449.0, 127.0, 128.0, 0.875, 0.9921875, 0.9999, 463.9, 464.0]
    g = torch.Generator().manual_seed(1)
    n, dim = len(tops), 64
    rows = []
    for t in tops:
        y = torch.rand(dim, generator=g, dtype=torch.float64) * 2 - 1
        y[0] = 1
        # ties between codes, and numbers below the least one
        y[1:8] = torch.tensor([17 / 256, 18.5 / 448, 9.5 / 127, 2.0 ** -19, 2.0 ** -18 * 1.5, -1.0, 0.0])
        rows.append(y * t)
    x = torch.stack(rows).float().to(dt)[:, None]
    odd = x.clone()
    odd[2, 0, 9], odd[3, 0, 10], odd[5, 0, 3], odd[6] = float("nan"), float("inf"), float("-inf"), float("nan")
    for r in (x, odd):
        cache = Q.Cache(n, 1, 1, dim, 1, code)
        dev = cache.tensors(DEV)
        table, cu, seq = i32(torch.arange(n)[:, None]), i32(torch.arange(n + 1)), i32([1] * n)
        print("edges", code, dt, flush=True)
        P8.kv_append_q8(r.to(DEV), r.flip(2).contiguous().to(DEV), *dev, table, cu, seq)
        torch.cuda.synchronize()
        cache.append(r, r.flip(2), table.cpu(), np.arange(n + 1), [1] * n)
        assert cache.same(dev)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("block", [16, 32, 64])
def test_long_blocks_and_rows_past_the_registers(code, block):
    """More rows of a block than a unit of work holds, one joining, and a grown scale with many
    earlier rows."""
    page, hkv, dim = 64 if block < 64 else 192, 2, 128
    block = block if block < 64 else 192
    g = torch.Generator().manual_seed(block)
    table = torch.tensor([[1, 0, 3], [5, 2, 4]], dtype=torch.int32)
    cache = Q.Cache(6, hkv, page, dim, block, code)
    dev = cache.tensors(DEV)
    seq = [0, 0]
    for new, size in (([150, 191], 0.1), ([1, 0], 50.0), ([9, 1], 3.0), ([0, 100], 4000.0), ([20, 60], 1.0)):
        new = [min(t, 3 * page - s) for t, s in zip(new, seq)]
        seq = [s + t for s, t in zip(seq, new)]
        k, v = ((size * torch.randn(sum(new), hkv, dim, generator=g)).to(BF) for _ in range(2))
        cu = [0] + list(np.cumsum(new))
        print("long blocks", code, block, new, flush=True)
        P8.kv_append_q8(k.to(DEV), v.to(DEV), *dev, table.to(DEV), i32(cu), i32(seq))
        torch.cuda.synchronize()
        cache.append(k, v, table, cu, seq)
        assert cache.same(dev)


@pytest.mark.parametrize("code", CODES)
def test_rows_without_a_place_are_skipped(code):
    """Positions below 0, table entries that are no page, positions past the table, rows behind the
    last request, empty requests; read back, they are zeros."""
    page, block, hkv, dim, cols = 16, 8, 2, 64, 3
    table = torch.tensor([[2, -1, 4], [99, 5, 6], [0, 1, 3], [7, 8, 9], [-5, -1, 2 ** 30]], dtype=torch.int32)
    new, seq = [20, 30, 0, 9, 5], [46, 70, 10, 4, 40]      # past the table, in holes, below 0
    cu = [0] + list(np.cumsum(new))
    g = torch.Generator().manual_seed(5)
    T = cu[-1] + 6
    k, v = (torch.randn(T, hkv, dim, generator=g).to(BF) for _ in range(2))
    cache = Q.Cache(10, hkv, page, dim, block, code, scale=2.0)
    dev = cache.tensors(DEV)
    print("no place", code, flush=True)
    P8.kv_append_q8(k.to(DEV), v.to(DEV), *dev, table.to(DEV), i32(cu), i32(seq))
    ko, vo = P8.kv_read_q8(*dev, table.to(DEV), i32(cu), i32(seq), total_tokens=T, dtype=FP)
    torch.cuda.synchronize()
    cache.append(k, v, table, cu, seq)
    assert cache.same(dev)
    for i, t in enumerate(new):
        for x in range(t):
            p = seq[i] - t + x
            pg = int(table[i, p // page]) if 0 <= p < cols * page else -1
            for side, out in ((0, ko), (1, vo)):
                want = cache.row(side, pg, p % page) if 0 <= pg < 10 else np.zeros((hkv, dim))
                assert np.array_equal(out[cu[i] + x].cpu().double().numpy(), want, equal_nan=True), (i, p)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dt", [BF, FP])
def test_append_and_read_of_strided_rows_and_pools(code, dt):
    """K and V rows of one projection, K and V pages of one pool, a slice of a wider table."""
    page, block, hkv, dim, T = 16, 16, 2, 64, 41
    g = torch.Generator().manual_seed(8)
    proj = torch.randn(T, 3 * hkv, dim, generator=g).to(dt)
    wide = torch.full((2, 9), -1, dtype=torch.int32)
    wide[:, 2:5] = torch.tensor([[0, 3, 5], [1, 4, 2]])
    cu, seq = [0, 30, 41], [30, 11]
    cache = Q.Cache(6, hkv, page, dim, block, code, scale=1.0)
    kc, vc, ks, vs = cache.tensors(DEV)
    pool = torch.stack([kc.view(torch.uint8), vc.view(torch.uint8)], 1).view(kc.dtype)
    p, w = proj.to(DEV), wide.to(DEV)
    print("strided", code, dt, flush=True)
    P8.kv_append_q8(p[:, :hkv], p[:, 2 * hkv:], pool[:, 0], pool[:, 1], ks, vs, w[:, 2:5], i32(cu), i32(seq))
    ko, vo = P8.kv_read_q8(pool[:, 0], pool[:, 1], ks, vs, w[:, 2:5], torch.tensor(cu), i32(seq), dtype=FP)
    torch.cuda.synchronize()
    cache.append(proj[:, :hkv], proj[:, 2 * hkv:], wide[:, 2:5], cu, seq)
    assert cache.same((pool[:, 0].view(torch.uint8), pool[:, 1].view(torch.uint8), ks, vs))
    for side, out in ((0, ko), (1, vo)):
        for i in range(2):
            for x in range(cu[i], cu[i + 1]):
                pos = x - cu[i]
                assert np.array_equal(out[x].cpu().double().numpy(), cache.row(side, int(wide[i, 2 + pos // page]), pos % page))


@pytest.mark.parametrize("n", [63, 64, 65, 200, 256, 257, 3000])
def test_many_requests_and_offsets_that_decrease(n):
    """More requests than a wave looks through at once; offsets out of order write nothing wrong."""
    page, hkv, dim = 4, 1, 64
    g = torch.Generator().manual_seed(2)
    seq = torch.randint(0, 8, (n,), generator=g)
    new = torch.minimum(torch.randint(0, 3, (n,), generator=g), seq)
    cu = [0] + torch.cumsum(new, 0).tolist()
    table = torch.randperm(2 * n, generator=g).view(n, 2).to(torch.int32)
    k, v = (torch.randn(cu[-1], hkv, dim, generator=g).to(BF) for _ in range(2))
    cache = Q.Cache(2 * n, hkv, page, dim, 2, "e4m3", scale=1.0)
    dev = cache.tensors(DEV)
    print("many requests", flush=True)
    P8.kv_append_q8(k.to(DEV), v.to(DEV), *dev, table.to(DEV), i32(cu), seq.to(DEV))
    ko, _ = P8.kv_read_q8(*dev, table.to(DEV), i32(cu), seq.to(DEV), total_tokens=cu[-1])
    torch.cuda.synchronize()
    cache.append(k, v, table, cu, seq.tolist())
    assert cache.same(dev)
    own = torch.from_numpy(np.stack([cache.row(0, int(table[i, p // page]), p % page)
                                     for i in range(n) for p in range(int(seq[i] - new[i]), int(seq[i]))]))
    assert torch.equal(ko.cpu(), own.to(BF))
    bad = torch.tensor([0, 40, 10, 90, cu[-1] + 50], dtype=torch.int32, device=DEV)
    P8.kv_append_q8(k.to(DEV), v.to(DEV), *dev, table[:4].to(DEV), bad, i32([8] * 4))
    P8.kv_read_q8(*dev, table[:4].to(DEV), bad, i32([8] * 4), total_tokens=cu[-1])
    torch.cuda.synchronize()


@pytest.mark.parametrize("page,pages", [(16, 1 << 21), (1 << 25, 3)])
def test_cache_offsets_past_32_bits(page, pages):
    """A pool of 2^25 tokens of 2 heads and more, of which a step writes, reads and attends to the end."""
    dim, hkv, window, sinks, new = 64, 2, 70, 3, 40
    L = page * pages // 2 if page > 16 else 4000
    g = torch.Generator().manual_seed(1)
    print("offsets", page, pages, flush=True)
    codes = [torch.empty(pages, hkv, page, dim, dtype=torch.int8, device=DEV).view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.empty(pages, hkv, page // 8, device=DEV) for _ in range(2)]
    cols = -(-L // page)
    table = (pages - 1 - torch.arange(cols, device=DEV)).to(torch.int32)[None]
    for m, at in ((8, 8), (128, L)):        # the sinks, then the end
        k, v = (torch.randn(m, hkv, dim, generator=g).to(BF) for _ in range(2))
        P8.kv_append_q8(k.to(DEV), v.to(DEV), *codes, *scales, table, i32([0, m]), i32([at]))
        kr, vr = P8.kv_read_q8(*codes, *scales, table, i32([0, m]), i32([at]), total_tokens=m, dtype=FP)
        torch.cuda.synchronize()
        # half a step of e4m3 (2^-4 of the value, or 2^-10 of the scale where it is below its normal numbers)
        for x, y in ((k, kr), (v, vr)):
            assert torch.all((y.cpu() - x.float()).abs() <= 2.0 ** -4 * x.float().abs() + 2.0 ** -10 * x.float().abs().max() / 224)
        if m == 8:
            first = kr[:sinks].cpu(), vr[:sinks].cpu()
    keys = torch.cat([first[0], kr.cpu()])
    values = torch.cat([first[1], vr.cpu()])
    key_pos = torch.cat([torch.arange(sinks), torch.arange(L - 128, L)])
    q = torch.randn(new, hkv, dim, generator=g).to(BF)
    for t in (new, 1):
        out = P8.paged_attention_q8(q[:t].to(DEV), *codes, *scales, table, i32([0, t]), i32([L]), window=window,
                                    sinks=sinks).cpu().double()
        for x in range(t):
            pos = L - t + x
            see = (key_pos <= pos) & ((pos - key_pos < window) | (key_pos < sinks))
            for h in range(hkv):
                s = dim ** -0.5 * (keys[see, h].double() @ q[x, h].double())
                ref = torch.softmax(s, 0) @ values[see, h].double()
                # a probability and the output are each rounded by at most 2^-8 of their size
                tol = 1.01 * 2.0 ** -8 * (values[see, h].double().abs().max() + ref.abs())
                assert torch.all((out[x, h] - ref).abs() <= tol), (t, x)


# ------------------------------------------------------------------ attention

def attend(c, cache, window=0, sinks=0, scale=None, **kw):
    """The operator on the case's tensors, every output pre-filled."""
    print(f"attend_q8 q={tuple(c.q.shape)} page={cache.page} block={cache.block} {cache.code} {c.q.dtype} "
          f"window={window} sinks={sinks} {kw}", flush=True)
    out = torch.full(c.q.shape, 7.0, dtype=c.q.dtype, device=DEV)
    lse = torch.full(c.q.shape[:2], 7.0, dtype=FP, device=DEV)
    P8.paged_attention_q8(c.q.to(DEV), *cache.tensors(DEV), c.table.to(DEV), c.cu.to(DEV), c.seq.to(DEV),
                          scale=scale, window=window, sinks=sinks, output=out, lse=lse, **kw)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu()


SMALL = {k: v for k, v in CASES.items() if v[6] != FP}
BLOCKS = {1: 1, 3: 3, 16: 8, 32: 32, 48: 24, 64: 16, 512: 128}


@pytest.mark.parametrize("name", list(SMALL))
@pytest.mark.parametrize("splits", [0, 1, 5])
@pytest.mark.parametrize("code", CODES)
def test_attention_matches_64_bits(name, splits, code):
    ctx, new, hq, hkv, dim, page, dt, window, sinks = SMALL[name]
    c, cache = Q.make(ctx, new, hq, hkv, dim, page, BLOCKS[page], dt, code, seed=len(name), pad_rows=3)
    hint = max(new) if splits != 5 else None
    check(c, page, attend(c, cache, window, sinks, splits=splits, max_new_len=hint), window, sinks)


@pytest.mark.parametrize("page,block", [(16, 16), (16, 1), (20, 5), (7, 7), (64, 32), (128, 128), (24, 3)])
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("new", [[1, 1, 1], [3, 8, 1], [90, 1, 130]])
@pytest.mark.parametrize("code", CODES)
def test_attention_over_any_page_and_block(page, block, dt, new, code):
    dim = 64 if page in (20, 64) else 128
    c, cache = Q.make([200, 31, 0], new, 4, 2, dim, page, block, dt, code, seed=page + block, pad_rows=1)
    check(c, page, attend(c, cache, splits=2))
    if page == 16:
        check(c, page, attend(c, cache, 50, 3), 50, 3)


WIDE = {
    # context, new, hq, hkv, dim, page, block, window, sinks: tiles of eight waves (by width) and of four
    "long_table": ([300], [600], 8, 1, 128, 64, 64, 0, 0),
    "ragged": ([0, 70, 5], [300, 1, 513], 6, 2, 64, 48, 16, 0, 0),
    "window": ([500, 0], [200, 260], 4, 1, 128, 16, 16, 100, 5),
}


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("name", list(WIDE))
def test_chunks_match_64_bits(name, code, dt):
    ctx, new, hq, hkv, dim, page, block, window, sinks = WIDE[name]
    c, cache = Q.make(ctx, new, hq, hkv, dim, page, block, dt, code, seed=3)
    rows = set(range(0, 40)) | set(range(int(c.cu[-1]) - 45, int(c.cu[-1]))) | set(range(100, 600, 37))
    out, lse = attend(c, cache, window, sinks)
    ref, rl, tol, tl = R.attention(c, page, dim ** -0.5, window, sinks, rows=rows)
    for x in sorted(rows & set(range(int(c.cu[-1])))):
        assert np.all(np.abs(out[x].double().numpy() - ref[x]) <= tol[x]), x
        assert np.all(np.abs(lse[x].double().numpy() - rl[x]) <= tl[x]), x


def eight_waves(code, dim, dt):
    """A case that takes the tiles of eight waves: a wide table and many rows; few keys exist."""
    hq, hkv, page, block, new = 64, 2, 64, 16, 1100
    c, cache = Q.make([200], [new], hq, hkv, dim, page, block, dt, code, seed=4)
    table = torch.full((1, 600), -1, dtype=torch.int32)
    table[:, :c.table.shape[1]] = c.table
    c.table = table
    return c, cache


@pytest.mark.parametrize("dim,dt", [(128, BF), (64, HF)])
@pytest.mark.parametrize("code", CODES)
def test_tiles_of_eight_waves(code, dim, dt):
    c, cache = eight_waves(code, dim, dt)
    rows = {0, 1, 31, 500, 777, 1098, 1099}
    for splits in (0, 1, 4):
        out, lse = attend(c, cache, splits=splits)
        ref, rl, tol, tl = R.attention(c, cache.page, dim ** -0.5, rows=rows)
        for x in rows:
            assert np.all(np.abs(out[x].double().numpy() - ref[x]) <= tol[x]), x
            assert np.all(np.abs(lse[x].double().numpy() - rl[x]) <= tl[x]), x


@pytest.mark.parametrize("dim,dt,cols", [(128, BF, 0), (64, HF, 0), (128, BF, 520)])
@pytest.mark.parametrize("code", CODES)
def test_ragged_requests_cut_into_pieces(code, dim, dt, cols):
    # rows for 256 workgroups and keys for two pieces; a wide table's take eight waves and more pieces
    c, cache = Q.make([3600, 60, 1700], [500, 90, 500], 32, 8, dim, 64, 32, dt, code, seed=6, pad_rows=2)
    if cols:
        table = torch.full((3, cols), -1, dtype=torch.int32)
        table[:, :c.table.shape[1]] = c.table
        c.table = table
    nbytes = P8.paged_attention_q8_workspace_bytes(c.q.to(DEV), *cache.tensors(DEV), c.table.to(DEV))
    assert nbytes > 0       # it is cut
    rows = {0, 63, 255, 499, 500, 589, 590, 811, 1089}
    out, lse = attend(c, cache)
    ref, rl, tol, tl = R.attention(c, cache.page, dim ** -0.5, rows=rows)
    for x in rows:
        assert np.all(np.abs(out[x].double().numpy() - ref[x]) <= tol[x]), x
        assert np.all(np.abs(lse[x].double().numpy() - rl[x]) <= tl[x]), x
    assert torch.all(out[1090:] == 7.0) and torch.all(lse[1090:] == 7.0)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("ctx,new,window,sinks", [
    (40, 3, 0, 0), (40, 30, 0, 0), (100, 90, 24, 3), (300, 200, 0, 0), (0, 300, 70, 5), (90, 6, 20, 3)])
def test_nan_codes_stay_where_they_are_seen(dt, ctx, new, window, sinks):
    page = 16
    c, cache = Q.make([ctx], [new], 4, 2, 128, page, 8, dt, "e4m3", seed=9)
    L = ctx + new
    for pos, side in ((L - 1, 1), (L - 2, 0), (L // 2, 1)):
        pg = int(c.table[0, pos // page])
        cache.codes[side][pg, 0, pos % page, 5] = 0x7f
        (c.keys, c.values)[side][0][pos, 0, 5] = float("nan")
    out, _ = attend(c, cache, window, sinks)
    with np.errstate(all="ignore"):
        ref, _, tol, _ = R.attention(c, page, 128 ** -0.5, window, sinks)
    o = out.double().numpy()
    fine = np.isfinite(ref)
    assert np.array_equal(np.isfinite(o), fine)
    assert np.all(np.abs(o[fine] - ref[fine]) <= tol[fine])


@pytest.mark.parametrize("what", [float("nan"), float("inf"), 0.0, -1.0])
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dt,new", [(BF, 4), (BF, 100), (HF, 7), (HF, 150)])
def test_a_hidden_blocks_scale_reaches_no_row(code, dt, new, what):
    """The last block, which only the last rows see, has a bad scale: the others stay within the
    tolerance of the definition.  (Their bits may change: a tile that a hidden value spoils is summed once
    more key by key, in fp32 as the matrix instructions do but in another order.)"""
    c, cache = Q.make([60], [new], 4, 2, 128, 16, 4, dt, code, seed=10)
    last = 60 + new - 1
    first = last // 4 * 4
    ref, rl, tol, tl = R.attention(c, 16, 128 ** -0.5)
    pg = int(c.table[0, last // 16])
    for s in cache.scales:
        s[pg, :, last % 16 // 4] = what
    out, lse = attend(c, cache)
    rows = first - 60                       # rows whose position is before the block
    assert np.all(np.abs(out.double().numpy() - ref)[:rows] <= tol[:rows])
    assert np.all(np.abs(lse.double().numpy() - rl)[:rows] <= tl[:rows])


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dt,new", [(BF, 1), (BF, 60), (HF, 9), (HF, 200)])
def test_missing_pages_hold_no_key(code, dt, new):
    c, cache = Q.make([40, 100], [new, new], 4, 2, 128, 16, 16, dt, code, seed=6,
                      holes=[(0, 1), (1, 0), (1, 3)])
    check(c, 16, attend(c, cache))
    check(c, 16, attend(c, cache, 30, 2), 30, 2)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("new", [1, 50])
def test_lengths_below_the_new_tokens_and_past_the_table(code, new):
    c, cache = Q.make([0, 30], [new, new], 2, 1, 64, 16, 8, BF, code, seed=7)
    c.seq[0] = new - 1                        # the first row lies below position 0
    c.keys[0], c.values[0] = c.keys[0][:new - 1], c.values[0][:new - 1]
    check(c, 16, attend(c, cache))


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("code", CODES)
def test_more_new_tokens_than_the_hint_says(code, dt):
    """A hint of one new token for chunks: the rows of a request in turns of 16, hidden NaN codes kept out."""
    c, cache = Q.make([100, 0, 7], [70, 33, 1], 4, 2, 128, 16, 8, dt, code, seed=14)
    check(c, 16, attend(c, cache, max_new_len=1))
    check(c, 16, attend(c, cache, 40, 3, max_new_len=1, splits=3), 40, 3)
    if code == "e4m3":
        for i, pos, side in ((0, 169, 1), (0, 120, 1), (1, 32, 0)):
            cache.codes[side][int(c.table[i, pos // 16]), 1, pos % 16, 77] = 0xff
            (c.keys, c.values)[side][i][pos, 1, 77] = float("nan")
        out, _ = attend(c, cache, max_new_len=1)
        with np.errstate(all="ignore"):
            ref, _, tol, _ = R.attention(c, 16, 128 ** -0.5)
        o = out.double().numpy()
        fine = np.isfinite(ref)
        assert np.array_equal(np.isfinite(o), fine)
        assert np.all(np.abs(o[fine] - ref[fine]) <= tol[fine])


def test_scales_far_apart_and_tiny():
    """Blocks whose values differ by 2^60, and values near the least normal number of fp32."""
    for dt, sizes in ((BF, [2.0 ** -60, 1.0, 2.0 ** 30]), (BF, [2.0 ** -100, 2.0 ** -90, 2.0 ** -95]),
                      (HF, [2.0 ** -6, 1.0, 2.0 ** 8])):
        for new in (1, 70):
            c, cache = Q.make([50], [new], 4, 2, 128, 16, 16, dt, "e4m3", seed=12)
            for b in range(-(-(50 + new) // 16)):
                z = sizes[b % 3]
                pg = int(c.table[0, b])
                cache.scales[1][pg] *= z
                c.values[0][16 * b:16 * b + 16] *= z
            check(c, 16, attend(c, cache))


def test_strides_and_views():
    """q inside a fused projection, K and V as halves of one pool, a slice of a wider table."""
    for new in (1, 40):
        c, cache = Q.make([70, 9], [new, new], 4, 2, 128, 16, 8, BF, "e4m3", seed=5)
        T = c.q.shape[0]
        proj = torch.full((T, 12, 128), float("nan"), dtype=BF)
        proj[:, 4:8] = c.q
        kc, vc, ks, vs = cache.tensors(DEV)
        pool = torch.stack([kc.view(torch.uint8), vc.view(torch.uint8)], 1).view(kc.dtype)
        wide = torch.full((2, c.table.shape[1] + 5), -1, dtype=torch.int32)
        wide[:, 2:2 + c.table.shape[1]] = c.table
        out, lse = P8.paged_attention_q8(proj.to(DEV)[:, 4:8], pool[:, 0], pool[:, 1], ks, vs,
                                         wide.to(DEV)[:, 2:2 + c.table.shape[1]], c.cu.to(DEV), c.seq.to(DEV),
                                         return_lse=True)
        torch.cuda.synchronize()
        check(c, 16, (out.cpu(), lse.cpu()))


def test_calls_without_tokens_requests_or_pages():
    c, cache = Q.make([20], [5], 2, 1, 64, 16, 16, BF, "int8", seed=1)
    kc, vc, ks, vs = cache.tensors(DEV)
    empty = torch.zeros(0, 2, 64, dtype=BF, device=DEV)
    none = torch.zeros(0, 3, dtype=torch.int32, device=DEV)
    assert P8.paged_attention_q8(empty, kc, vc, ks, vs, c.table.to(DEV), i32([0, 0]), c.seq.to(DEV)).shape == (0, 2, 64)
    q = c.q.to(DEV)
    out = torch.full_like(q, 4)
    P8.paged_attention_q8(q, kc, vc, ks, vs, none, i32([0]), i32([]), output=out)
    assert torch.all(out == 4)
    out = P8.paged_attention_q8(q, kc, vc, ks, vs, torch.zeros(1, 0, dtype=torch.int32, device=DEV), i32([0, 5]), c.seq.to(DEV))
    assert torch.all(out == 0)
    before = [t.clone().view(torch.uint8) for t in (kc, vc, ks, vs)]
    rows = torch.ones(5, 1, 64, dtype=BF, device=DEV)
    P8.kv_append_q8(rows[:0], rows[:0], kc, vc, ks, vs, c.table.to(DEV), i32([0, 0]), c.seq.to(DEV))
    P8.kv_append_q8(rows, rows, kc, vc, ks, vs, none, i32([0]), i32([]))
    P8.kv_append_q8(rows, rows, kc, vc, ks, vs, torch.zeros(1, 0, dtype=torch.int32, device=DEV), i32([0, 5]), c.seq.to(DEV))
    k0, v0 = P8.kv_read_q8(kc, vc, ks, vs, torch.zeros(1, 0, dtype=torch.int32, device=DEV), i32([0, 5]), c.seq.to(DEV), total_tokens=5)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b.view(torch.uint8)) for a, b in zip(before, (kc, vc, ks, vs)))
    assert torch.all(k0 == 0) and torch.all(v0 == 0)


# ------------------------------------------------------------------- together

def test_streams_equal_bits_and_given_workspaces():
    c, cache = Q.make([1500, 3], [1, 1], 8, 2, 128, 16, 16, BF, "e4m3", seed=31)
    args = [c.q.to(DEV), *cache.tensors(DEV), c.table.to(DEV), c.cu.to(DEV), c.seq.to(DEV)]
    ref = P8.paged_attention_q8(*args, splits=4)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(P8.paged_attention_q8(*args, splits=4))
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
    need = P8.paged_attention_q8_workspace_bytes(*args[:6], splits=4)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    assert torch.equal(P8.paged_attention_q8(*args, splits=4, workspace=ws), ref)
    with pytest.raises(ValueError, match="workspace"):
        P8.paged_attention_q8(*args, splits=4, workspace=ws[:64])


@pytest.mark.parametrize("code", CODES)
def test_steps_of_a_batch(code):
    """Prefill, then decode steps with a rejected draft: tables, rotary positions, the append and the
    attention together, each step's attention against the plain form over what the cache stands for, and
    that against the rows to within half a step of the codes."""
    hq, hkv, dim, page, block, dt = 4, 2, 128, 16, 8, BF
    steps = [[37, 5, 70], [4, 1, 0], [2, 1, 3], [1, 1, 1]]
    rejected = [[0, 0, 0], [3, 0, 0], [0, 0, 2], [0, 0, 0]]
    n, num_pages = 3, 14
    g = torch.Generator().manual_seed(1)
    table = torch.full((n, 7), -1, dtype=torch.int32, device=DEV)
    free = torch.randperm(num_pages, generator=g).to(torch.int32).to(DEV)
    cache = Q.Cache(num_pages, hkv, page, dim, block, code)
    dev = cache.tensors(DEV)
    f = positions.rotary_frequencies(dim).to(DEV)
    ctx = torch.zeros(n, dtype=torch.int32, device=DEV)
    for s, new in enumerate(steps):
        T = sum(new) + 2
        q, k, v = (torch.randn(T, h, dim, generator=g).to(dt) for h in (hq, hkv, hkv))
        print("step", code, s, flush=True)
        t = paged.page_tables(ctx, i32(new), free, table, page, num_pages, max_tokens=T)
        qd, kd = q.to(DEV), k.to(DEV)
        positions.rotary(qd, kd, t.positions, f, q_out=qd, k_out=kd)
        P8.kv_append_q8(kd, v.to(DEV), *dev, table, t.cu_seqlens, t.seq_lens)
        out = P8.paged_attention_q8(qd, *dev, table, t.cu_seqlens, t.seq_lens)
        torch.cuda.synchronize()
        cache.append(kd.cpu(), v, table.cpu(), t.cu_seqlens.tolist(), t.seq_lens.tolist())
        assert cache.same(dev)
        seq = t.seq_lens.tolist()
        rows = [[torch.from_numpy(np.stack([cache.row(side, int(table[i, p // page]), p % page) for p in range(m)]))
                 for i, m in enumerate(seq)] for side in (0, 1)]
        c = R.Case(qd.cpu(), torch.from_numpy(cache.codes[0]), None, table.cpu(), t.cu_seqlens.cpu(), t.seq_lens.cpu(),
                   rows[0], rows[1])
        ref, _, tol, _ = R.attention(c, page, dim ** -0.5)
        m = sum(new)
        assert np.all(np.abs(out.double().cpu().numpy() - ref)[:m] <= tol[:m])
        free = free[int(t.pages_taken):].contiguous()
        ctx = t.seq_lens - i32(rejected[s])
        # the pages of rejected positions stay in the table: the next step's tables take new ones
        # only past those that its lengths need, so give back what they no longer do
        have = -(-ctx // page)
        for i in range(n):
            extra = table[i, int(have[i]):]
            free = torch.cat([extra[extra >= 0], free])
            extra.fill_(-1)


def test_captured_steps_replay_as_the_eager_ones():
    """Tables, rotary, append, read and attention captured once, with shared scratch in two graphs,
    replayed in turn on new lengths and rows, with eager steps between."""
    from test_graphs_gpu import capture
    hq, hkv, dim, page, block, n, num_pages, T = 4, 2, 64, 16, 4, 5, 60, 40
    g = torch.Generator().manual_seed(2)
    ids = torch.randperm(num_pages, generator=g).to(torch.int32).to(DEV)
    table0 = torch.cat([ids[:30].reshape(5, 6), torch.full((5, 4), -1, dtype=torch.int32, device=DEV)], 1)
    free = ids[30:].contiguous()
    f = positions.rotary_frequencies(dim).to(DEV)
    sides = []
    ws = None
    for code in CODES:
        start = [t.to(DEV) for t in Q.make([90] * 5, [1] * 5, hq, hkv, dim, page, block, BF, code, seed=3)[1].tensors()]
        start = [torch.cat([t.view(torch.uint8)] * 2)[:num_pages].view(t.dtype) if t.dtype != FP else
                 torch.ones(num_pages, hkv, page // block, device=DEV) for t in start]
        ins = [torch.zeros(n, dtype=torch.int32, device=DEV) for _ in range(2)] + \
              [torch.zeros(T, h, dim, dtype=BF, device=DEV) for h in (hq, hkv, hkv)]
        room = paged.PageTables(*[torch.zeros(m, dtype=d, device=DEV) for m, d in (
            (n + 1, torch.int32), (n, torch.int32), (T, torch.int64), (T, torch.int32), (1, torch.int32))])
        outs = [torch.zeros(T, h, dim, dtype=BF, device=DEV) for h in (hq, hkv, hkv)]
        if ws is None:
            ws = torch.empty(P8.paged_attention_q8_workspace_bytes(ins[2], *start, table0, splits=4),
                             dtype=torch.uint8, device=DEV)

        def run(ins, cache, table, room, outs):
            paged.page_tables(ins[0], ins[1], free, table, page, num_pages, out=room)
            positions.rotary(ins[2], ins[3], room.positions, f, q_out=ins[2], k_out=ins[3])
            P8.kv_append_q8(ins[3], ins[4], *cache, table, room.cu_seqlens, room.seq_lens)
            P8.paged_attention_q8(ins[2], *cache, table, room.cu_seqlens, room.seq_lens, output=outs[0], splits=4,
                                  workspace=ws)
            P8.kv_read_q8(*cache, table, room.cu_seqlens, room.seq_lens, k_out=outs[1], v_out=outs[2])

        cache, table = [t.clone() for t in start], table0.clone()
        graph = capture(lambda: run(ins, cache, table, room, outs))
        sides.append((start, ins, room, outs, cache, table, graph, run))
    for r in range(5):
        for start, ins, room, outs, cache, table, graph, run in (sides if r % 2 else sides[::-1]):
            lens, news = torch.randint(0, 90, (n,), generator=g), torch.randint(0, 8, (n,), generator=g)
            fresh = [lens, news] + [torch.randn(T, h, dim, generator=g) for h in (hq, hkv, hkv)]
            for dst, src in zip(ins, fresh):
                dst.copy_(src.to(DEV))
            for dst, src in zip(cache + [table], start + [table0]):
                dst.copy_(src)
            eager = ([x.clone() for x in ins], [x.clone() for x in start], table0.clone(),
                     paged.PageTables(*[x.clone() for x in room]), [torch.full_like(o, 3) for o in outs])
            for o in outs:
                o.fill_(3)
            print("replay", r, flush=True)
            run(*eager)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(outs + cache + [table], eager[4] + eager[1] + [eager[2]]):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("new", [1, 3, 6, 100])
@pytest.mark.parametrize("ctx,window,sinks", [(300, 0, 0), (420, 200, 80)])
def test_a_seen_nan_outlives_far_larger_scores(dt, new, ctx, window, sinks):
    """A NaN code of V at an early key that every row sees, and keys behind it, of the same wave, whose scores
    are hundreds above: one token, drafts of up to 16 and up to 32 rows, and chunks agree that it is seen."""
    c, cache = Q.make([ctx], [new], 8, 2, 128, 16, 8, dt, "e4m3", seed=21)
    big = 64            # keys 64 .. 71, a block, have K values 2^8 times as large
    cache.scales[0][int(c.table[0, big // 16]), :, big % 16 // 8] *= 256.0
    c.keys[0][big:big + 8] *= 256.0
    for pos in (5, ctx + new - 1):      # seen by all rows, and by the last token's alone
        cache.codes[1][int(c.table[0, pos // 16]), 0, pos % 16, 7] = 0x7f
        c.values[0][pos, 0, 7] = float("nan")
    out, _ = attend(c, cache, window, sinks)
    with np.errstate(all="ignore"):
        ref, _, tol, _ = R.attention(c, 16, 128 ** -0.5, window, sinks)
    o = out.double().numpy()
    fine = np.isfinite(ref)
    assert np.array_equal(np.argwhere(~fine)[:, 2], np.full(new * 4, 7))    # the four heads on K head 0
    assert np.array_equal(np.isfinite(o), fine)
    assert np.all(np.abs(o[fine] - ref[fine]) <= tol[fine])


# In [1, 2), the number before 2 among them: a scale times one has the same exponent.
WITHIN = torch.tensor([1.0, 1.25, 1.5, 2.0 - 2.0 ** -23])


def within(scales, seed):
    """Scales that are not powers of two, with the exponents of these."""
    g = torch.Generator().manual_seed(seed)
    return scales * WITHIN[torch.randint(0, 4, scales.shape, generator=g)].to(scales.device)


def exponents(scales):
    return scales.cpu().view(torch.int32) & 0x7f800000


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dim,dt", [(128, BF), (64, HF)])
@pytest.mark.parametrize("new", [1, 3, 7, 90])
def test_scales_count_by_their_exponents_in_attention(code, dim, dt, new):
    """Scales that are not powers of two give, bit by bit, what the powers of two below them give: over K
    and V, in a single token, short drafts, 28 rows and chunks."""
    c, cache = Q.make([200, 31], [new, new], 8, 2, dim, 16, 4, dt, code, seed=30 + new)
    kc, vc, ks, vs = cache.tensors(DEV)
    args = c.table.to(DEV), c.cu.to(DEV), c.seq.to(DEV)
    print("exponents", code, dim, dt, new, flush=True)
    for odd_k, odd_v in ((True, False), (False, True)):
        o = P8.paged_attention_q8(c.q.to(DEV), kc, vc, within(ks, 1) if odd_k else ks, within(vs, 2) if odd_v else vs,
                                  *args, return_lse=True, max_new_len=new)
        p = P8.paged_attention_q8(c.q.to(DEV), kc, vc, ks, vs, *args, return_lse=True, max_new_len=new)
        torch.cuda.synchronize()
        assert torch.equal(o[0], p[0]) and torch.equal(o[1], p[1]), (odd_k, odd_v)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dt", [BF, HF, FP])
def test_scales_count_by_their_exponents_in_reads(code, dt):
    c, cache = Q.make([70, 9], [1, 1], 2, 2, 64, 16, 4, dt, code, seed=40)
    kc, vc, ks, vs = cache.tensors(DEV)
    cu = i32([0] + list(np.cumsum(c.seq.tolist())))
    print("exponents", code, dt, flush=True)
    got = [P8.kv_read_q8(kc, vc, *s, c.table.to(DEV), cu, c.seq.to(DEV), total_tokens=int(cu[-1]), dtype=dt)
           for s in ((ks, vs), (within(ks, 3), within(vs, 4)))]
    torch.cuda.synchronize()
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("page,block", [(16, 4), (48, 24), (128, 128)])
def test_scales_count_by_their_exponents_in_appends(code, page, block):
    """Rows that join a block keep the power of two or raise it, and leave a power of two there; blocks
    without new rows keep what they hold."""
    ctx, n = [70, 9, 33], 3
    c, cache = Q.make(ctx, [2] * n, 2, 2, 64, page, block, BF, code, seed=50)
    plain = cache.tensors(DEV)
    odd = [t.clone() for t in plain[:2]] + [within(s, i) for i, s in enumerate(plain[2:])]
    before = [s.clone() for s in odd[2:]]
    touched = torch.zeros(plain[2].shape, dtype=torch.bool)
    for i, t in enumerate(ctx):
        for p in (t, t + 1):
            touched[int(c.table[i, p // page]), :, p % page // block] = True
    g = torch.Generator().manual_seed(6)
    k, v = (torch.randn(2 * n, 2, 64, generator=g) for _ in range(2))
    k[2:] *= 1e-3                   # scales that stay
    v[:4] *= 1e3                    # and scales that grow
    k, v = k.to(BF).to(DEV), v.to(BF).to(DEV)
    print("exponents", code, page, block, flush=True)
    for cache in (plain, odd):
        P8.kv_append_q8(k, v, *cache, c.table.to(DEV), c.cu.to(DEV), c.seq.to(DEV))
    torch.cuda.synchronize()
    for side in (0, 1):
        assert torch.equal(plain[side].view(torch.uint8), odd[side].view(torch.uint8))
        p, o = plain[2 + side].cpu(), odd[2 + side].cpu()
        assert torch.equal(p[touched], o[touched])
        assert torch.equal(o[~touched].view(torch.int32), before[side].cpu()[~touched].view(torch.int32))
        assert torch.equal(exponents(o), exponents(p))


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_a_begun_block_without_a_scale_takes_the_rows(code, what):
    """Rows that start inside a block whose memory nobody has set: the scale is theirs."""
    page, block, hkv, dim = 16, 8, 2, 64
    g = torch.Generator().manual_seed(7)
    k, v = (torch.randn(3, hkv, dim, generator=g).to(BF) for _ in range(2))
    table, cu, seq = torch.tensor([[1, 0]], dtype=torch.int32), [0, 3], [6]
    cache = Q.Cache(2, hkv, page, dim, block, code, scale=1.0)
    dev = cache.tensors(DEV)
    for side in (0, 1):
        dev[2 + side][1, :, 0] = what
        cache.scales[side][1, :, 0] = 0.0       # below any that the rows need
        cache.codes[side][1, :, :3] = 0         # and rounded to zeros by it here
        dev[side].view(torch.uint8)[1, :, :3] = 0
    print("no scale", code, what, flush=True)
    P8.kv_append_q8(k.to(DEV), v.to(DEV), *dev, table.to(DEV), i32(cu), i32(seq))
    torch.cuda.synchronize()
    cache.append(k, v, table, cu, seq)
    assert cache.same(dev)


@pytest.mark.parametrize("dim,dt", [(128, BF), (64, HF)])
@pytest.mark.parametrize("code", CODES)
def test_tiles_of_eight_waves_cut_into_pieces(code, dim, dt):
    """Ragged requests whose rows fill the chip with workgroups of 256, over a wide table: eight waves, and
    visits of two pieces and three.  (A wide table alone does not take eight waves: 1092 tokens of 32 heads on 8
    make 144 such workgroups, and run on four.)  Over e4m3, with a NaN code too that one request's last token sees."""
    hq, hkv, cols = 64, 8, 520
    new = [600, 30, 430]
    c, cache = Q.make([4500, 9, 6300], new, hq, hkv, dim, 64, 32, dt, code, seed=8, pad_rows=2)
    table = torch.full((3, cols), -1, dtype=torch.int32)
    table[:, :c.table.shape[1]] = c.table
    c.table = table
    # 272 workgroups of 256 rows; pieces of 2048 keys at least, so 16 at most in 33280 (four waves: 15)
    rows, pieces = (sum(new) + 2) * hq, 16
    need = pieces * rows * dim * 4 + pieces * rows * 4 + rows * 4
    assert P8.paged_attention_q8_workspace_bytes(c.q, *cache.tensors(), c.table) == need
    look = {0, 63, 255, 599, 600, 629, 630, 811, 1058, 1059}
    for nan in ([False, True] if code == "e4m3" else [False]):
        if nan:
            pos = 4500 + 599
            cache.codes[1][int(c.table[0, pos // 64]), 3, pos % 64, 20] = 0xff
            c.values[0][pos, 3, 20] = float("nan")
        out, lse = attend(c, cache)
        with np.errstate(all="ignore"):
            ref, rl, tol, tl = R.attention(c, 64, dim ** -0.5, rows=look)
        o, fine = out.double().numpy(), np.isfinite(ref)
        assert np.count_nonzero(~fine) == (8 if nan else 0)     # the last token's eight heads on K head 3
        for x in sorted(look):
            f = fine[x]
            assert np.array_equal(np.isfinite(o[x]), f), x
            assert np.all(np.abs(o[x] - ref[x])[f] <= tol[x][f]), x
            assert np.all(np.abs(lse[x].double().numpy() - rl[x]) <= tl[x]), x
        assert torch.all(out[1060:] == 7.0) and torch.all(lse[1060:] == 7.0)


@pytest.mark.parametrize("n", [4, 64, 300])
@pytest.mark.parametrize("code", CODES)
def test_offsets_out_of_order_write_nothing_else(n, code):
    """Offsets that decrease, lie below 0 or past the rows: a block of the cache is what its request's rows make it
    or untouched, pages of no request are untouched, and so is what lies around the rows read."""
    page, block, hkv, dim, T = 8, 4, 2, 64, 210
    g = torch.Generator().manual_seed(n)
    cu = torch.sort(torch.randint(0, T + 1, (n + 1,), generator=g)).values
    swap = torch.randperm(n + 1, generator=g)[:max(2, n // 4)]
    cu[swap] = torch.randint(-50, T + 50, (swap.numel(),), generator=g)
    if n == 4:
        cu = torch.tensor([0, 40, 10, 90, T + 50])
    seq = torch.randint(0, 2 * page + 1, (n,), generator=g)
    pages = 4 * n
    table = torch.randperm(pages, generator=g)[:2 * n].view(n, 2).to(torch.int32)   # half of the pages
    k, v = (torch.randn(T, hkv, dim, generator=g).to(BF) for _ in range(2))
    cache = Q.Cache(pages, hkv, page, dim, block, code, scale=1.0)
    old = [x.copy() for x in cache.codes + cache.scales]
    dev = cache.tensors(DEV)
    print("out of order", n, code, flush=True)
    P8.kv_append_q8(k.to(DEV), v.to(DEV), *dev, table.to(DEV), i32(cu), i32(seq))
    torch.cuda.synchronize()
    cache.append(k, v, table, cu.clamp(0, T).tolist(), seq.tolist())
    shape = (pages, hkv, page // block, block * dim)
    made = 0
    for side in (0, 1):
        codes, scales = dev[side].cpu().view(torch.uint8).numpy().reshape(shape), dev[2 + side].cpu().numpy()
        is_old = (codes == old[side].reshape(shape)).all(-1) & (scales == old[2 + side])
        is_new = (codes == cache.codes[side].reshape(shape)).all(-1) & (scales == cache.scales[side])
        assert np.all(is_old | is_new)
        unlisted = np.setdiff1d(np.arange(pages), table.numpy())
        assert np.all(is_old[unlisted])
        made += int((~is_old).sum())
    assert made > 0
    room = [torch.full((T + 40, hkv, dim), 9.0, device=DEV) for _ in range(2)]
    P8.kv_read_q8(*dev, table.to(DEV), i32(cu), i32(seq), k_out=room[0][20:20 + T], v_out=room[1][20:20 + T])
    torch.cuda.synchronize()
    for x in room:
        assert torch.all(x[:20] == 9.0) and torch.all(x[20 + T:] == 9.0)
