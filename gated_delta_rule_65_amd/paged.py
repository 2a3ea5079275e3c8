"""ctypes binding of the paged attention operators (include/kda_paged.h).

The attention side of a hybrid model's serving step, beside the KDA layers of
``binding``: the step's block tables and slot maps (``page_tables``), the new key
and value rows into the paged cache (``kv_append``) and the attention over it
(``paged_attention``).  As in ``binding``, this layer checks and marshals arguments
only; every step of the computation runs in the library's HIP kernels, queued on
torch's current stream of the tensors' device.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import binding
from .binding import KDA_OK, _DTYPES, _need, _raise

_P, _I, _L, _Z, _F = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t,
                      ctypes.c_float)


class PageTablesArgs(ctypes.Structure):
    _fields_ = [
        ("struct_size", _Z),
        ("context_lens", _P), ("new_lens", _P), ("free_pages", _P), ("block_table", _P),
        ("table_stride", _L),
        ("n", _I), ("num_free", _I), ("max_pages", _I), ("page_size", _I), ("num_pages", _I),
        ("max_tokens", _L),
        ("slot_mapping", _P), ("positions", _P), ("cu_seqlens", _P), ("seq_lens", _P),
        ("pages_taken", _P), ("stream", _P),
    ]


class KvAppendArgs(ctypes.Structure):
    _fields_ = [
        ("struct_size", _Z),
        ("k", _P), ("v", _P), ("k_cache", _P), ("v_cache", _P), ("slot_mapping", _P),
        ("total_tokens", _L), ("k_stride", _L), ("v_stride", _L),
        ("k_page_stride", _L), ("v_page_stride", _L),
        ("dtype", _I), ("hkv", _I), ("head_dim", _I), ("page_size", _I), ("num_pages", _I),
        ("stream", _P),
    ]


class PagedAttentionArgs(ctypes.Structure):
    _fields_ = [
        ("struct_size", _Z),
        ("q", _P), ("k_cache", _P), ("v_cache", _P), ("block_table", _P), ("cu_seqlens", _P),
        ("seq_lens", _P), ("out", _P), ("lse", _P), ("workspace", _P), ("workspace_bytes", _Z),
        ("total_tokens", _L), ("q_stride", _L), ("k_page_stride", _L), ("v_page_stride", _L),
        ("table_stride", _L),
        ("dtype", _I), ("n", _I), ("hq", _I), ("hkv", _I),
        ("head_dim", _I), ("page_size", _I), ("num_pages", _I), ("max_pages", _I),
        ("window", _I), ("sinks", _I), ("max_new_len", _I), ("splits", _I),
        ("scale", _F), ("stream", _P),
    ]


_SIZEOF_TABLES = ctypes.sizeof(PageTablesArgs)
_SIZEOF_APPEND = ctypes.sizeof(KvAppendArgs)
_SIZEOF_ATTENTION = ctypes.sizeof(PagedAttentionArgs)

EXPORTS = ("kda_page_tables", "kda_kv_append", "kda_paged_attention_workspace_size",
           "kda_paged_attention")
# Workspace bytes that serve every paged_attention call (kda_paged.h).
PAGED_ATTENTION_WORKSPACE_MAX = (1 << 30) + (1 << 25)
_MAX_INT = 2**31 - 1     # ctypes cuts what an int32 field does not hold
_lib = None


def load_library():
    """The library with the paged entry points declared; raises if it is missing."""
    global _lib
    if _lib is None:
        lib = binding.load_library()
        P = ctypes.POINTER
        for name, args in (("kda_page_tables", [P(PageTablesArgs)]),
                           ("kda_kv_append", [P(KvAppendArgs)]),
                           ("kda_paged_attention", [P(PagedAttentionArgs)]),
                           ("kda_paged_attention_workspace_size",
                            [P(PagedAttentionArgs), P(ctypes.c_size_t)])):
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, ctypes.c_int
        _lib = lib
    return _lib


class PageTables(NamedTuple):
    """What page_tables computes beside the block table (device tensors)."""
    cu_seqlens: torch.Tensor     # int32 [n + 1]
    seq_lens: torch.Tensor       # int32 [n]
    slot_mapping: torch.Tensor   # int64 [max_tokens], -1 behind the last new token
    positions: torch.Tensor      # int32 [max_tokens], -1 behind the last new token
    pages_taken: torch.Tensor    # int32 [1]


# The checks below format their messages only when they fail: a call's host time is
# what a short decode step waits for.

def _fail(msg, exc=ValueError):
    raise exc(msg)


def _on_gpu(dev):
    if dev.type != "cuda":
        _fail(f"tensors must be on a GPU, got {dev}")


def _same_device(dev, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            _fail(f"{name} must be on {dev}")


# torch's own lookup of the current stream: 0.2 us, where building a Stream object to
# read its handle takes 1.9 of a short call's 8-12 us.  Builds without it take the object.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(dev):
    """The handle of torch's current stream on a GPU."""
    if _raw_stream is not None:
        return _raw_stream(dev.index)
    return torch.cuda.current_stream(dev).cuda_stream


def _call(fn, args, dev):
    """Runs a library call with the tensors' device current; raises on an error."""
    if dev.index is None or dev.index == torch.cuda.current_device():
        st = fn(ctypes.byref(args))
    else:
        with torch.cuda.device(dev):
            st = fn(ctypes.byref(args))
    if st != KDA_OK:
        _raise(binding.load_library(), st)


def _int32(x, n, name, dev):
    """A 1-D index tensor as a contiguous int32 one on dev."""
    if x.dim() != 1 or x.shape[0] != n:
        _fail(f"{name} must have shape [{n}]")
    if x.dtype is torch.int32 and x.device == dev and x.is_contiguous():
        return x
    if x.dtype is not torch.int32 and x.dtype is not torch.int64:
        _fail(f"{name} must have dtype torch.int32 or torch.int64", TypeError)
    return x.to(device=dev, dtype=torch.int32).contiguous()


def _table(block_table, n):
    """(row stride, columns) of an int32 [n, max_pages] block table."""
    if block_table.dim() != 2 or block_table.shape[0] != n:
        _fail(f"block_table must be [{n}, max_pages]")
    if block_table.dtype is not torch.int32:
        _fail("block_table must have dtype torch.int32", TypeError)
    cols = block_table.shape[1]
    if block_table.is_contiguous():
        return cols, cols
    if not ((cols == 1 or block_table.stride(1) == 1) and
            (n == 1 or block_table.stride(0) >= cols)):
        _fail("block_table rows must be dense")
    return (cols if n == 1 else block_table.stride(0)), cols


def _page_stride(name, cache):
    """Elements between pages of a [pages, Hkv, page_size, D] pool, 0 when dense.
    Pages may lie apart (K and V halves of one pool), each one is dense."""
    if cache.is_contiguous():
        return 0
    dense, msg = 1, f"{name}: each page must be a dense [Hkv, page_size, head_dim] block"
    for d in (3, 2, 1):
        _need(cache.shape[d] == 1 or cache.stride(d) == dense, msg)
        dense *= cache.shape[d]
    if cache.shape[0] == 1:
        return 0
    _need(cache.stride(0) >= dense, msg)
    return cache.stride(0)


def _pools(k_cache, v_cache, dtype, hkv, dim):
    """(K page stride, V page stride, page size, pages) of the caches."""
    shape = k_cache.shape
    if len(shape) != 4 or shape[1] != hkv or shape[3] != dim:
        _fail(f"k_cache must be [pages, {hkv}, page_size, {dim}]")
    if v_cache.shape != shape:
        _fail("v_cache must have k_cache's shape")
    if k_cache.dtype is not dtype or v_cache.dtype is not dtype:
        _fail(f"k_cache and v_cache must have dtype {dtype}", TypeError)
    return (_page_stride("k_cache", k_cache), _page_stride("v_cache", v_cache), shape[2], shape[0])


def page_tables(context_lens, new_lens, free_pages, block_table, page_size, num_pages,
                max_tokens=None, out=None):
    """A step's block tables and slot maps, built on the GPU from the requests'
    lengths (kda_page_tables).

    context_lens, new_lens [n]: cached and new tokens per request; free_pages [F]:
    page ids to take from, in order; block_table [n, max_pages] int32, updated in
    place (the entries of the pages taken; rows may lie apart); num_pages: pages of
    the cache.  max_tokens: room in the slot map, at least the step's new tokens (a
    captured step keeps its largest).  Returns a PageTables; ``out`` gives one to
    write into (its slot_mapping then sets max_tokens), none of it memory of an input:
    two that take turns serve steps that pass one's seq_lens on as context_lens."""
    if context_lens.dim() != 1:
        _fail("context_lens must be [n]")
    n = context_lens.shape[0]
    if free_pages.dim() != 1:
        _fail("free_pages must be [F]")
    stride, cols = _table(block_table, n)
    page_size, num_pages = int(page_size), int(num_pages)
    if not 1 <= page_size <= _MAX_INT:
        _fail("page_size must be >= 1 and below 2^31")
    if not 0 <= num_pages <= _MAX_INT:
        _fail("num_pages must be >= 0 and below 2^31")
    dev = block_table.device
    ctx = _int32(context_lens, n, "context_lens", dev)
    new = _int32(new_lens, n, "new_lens", dev)
    free = _int32(free_pages, free_pages.shape[0], "free_pages", dev)
    if out is None:
        if max_tokens is None or int(max_tokens) < 0:
            _fail("max_tokens is needed (the room for new tokens)")
        tokens = int(max_tokens)
        ints = torch.empty(2 * n + 2 + tokens, dtype=torch.int32, device=dev)
        cu, seq, taken, pos = ints.split_with_sizes((n + 1, n, 1, tokens))
        out = PageTables(cu, seq, torch.empty(tokens, dtype=torch.int64, device=dev), pos, taken)
    else:
        tokens = out.slot_mapping.shape[0]
        _need(max_tokens is None or int(max_tokens) == tokens,
              "max_tokens must be the length of out.slot_mapping")
        for name, t, shape, dt in (("cu_seqlens", out.cu_seqlens, (n + 1,), torch.int32),
                                   ("seq_lens", out.seq_lens, (n,), torch.int32),
                                   ("slot_mapping", out.slot_mapping, (tokens,), torch.int64),
                                   ("positions", out.positions, (tokens,), torch.int32),
                                   ("pages_taken", out.pages_taken, (1,), torch.int32)):
            if tuple(t.shape) != shape:
                _fail(f"out.{name} must have shape {list(shape)}")
            if t.dtype is not dt:
                _fail(f"out.{name} must have dtype {dt}", TypeError)
            if not t.is_contiguous():
                _fail(f"out.{name} must be contiguous")
            if t.device != dev:
                _fail(f"out.{name} must be on {dev}")
    _on_gpu(dev)
    lib = _lib or load_library()
    _call(lib.kda_page_tables, PageTablesArgs(
        _SIZEOF_TABLES, ctx.data_ptr(), new.data_ptr(), free.data_ptr(), block_table.data_ptr(),
        stride, n, free.shape[0], cols, page_size, num_pages, tokens,
        out.slot_mapping.data_ptr(), out.positions.data_ptr(), out.cu_seqlens.data_ptr(),
        out.seq_lens.data_ptr(), out.pages_taken.data_ptr(),
        _stream(dev)), dev)
    return out


def kv_append(k, v, k_cache, v_cache, slot_mapping):
    """Copies the rows k, v [T, Hkv, D] to their slots of the paged caches
    [pages, Hkv, page_size, D], in place (kda_kv_append).  slot_mapping [T] int64
    holds distinct slots page * page_size + offset; one outside the cache (-1) skips
    its token.  k and v may be views of a fused projection."""
    shape, dtype = k.shape, k.dtype
    if len(shape) != 3:
        _fail("k must be [T, Hkv, D]")
    if v.shape != shape:
        _fail("v must have k's shape")
    if dtype not in _DTYPES:
        _fail(f"unsupported dtype {dtype}", TypeError)
    if v.dtype is not dtype:
        _fail("v must have k's dtype", TypeError)
    T, hkv, dim = shape
    kp, vp, page_size, pages = _pools(k_cache, v_cache, dtype, hkv, dim)
    if slot_mapping.dim() != 1 or slot_mapping.shape[0] != T:
        _fail(f"slot_mapping must have shape [{T}]")
    if slot_mapping.dtype is not torch.int64:
        _fail("slot_mapping must have dtype torch.int64", TypeError)
    if not slot_mapping.is_contiguous():
        _fail("slot_mapping must be contiguous")
    ks, vs = _rows_stride("k", k), _rows_stride("v", v)
    dev = k.device
    if not (v.device == dev and k_cache.device == dev and v_cache.device == dev and
            slot_mapping.device == dev):
        _same_device(dev, v=v, k_cache=k_cache, v_cache=v_cache, slot_mapping=slot_mapping)
    _on_gpu(dev)
    lib = _lib or load_library()
    _call(lib.kda_kv_append, KvAppendArgs(
        _SIZEOF_APPEND, k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        slot_mapping.data_ptr(), T, ks, vs, kp, vp, _DTYPES[dtype], hkv, dim, page_size, pages,
        _stream(dev)), dev)


def _rows_stride(name, t):
    """Elements between the tokens of [T, H, D] rows, 0 when dense."""
    if t.is_contiguous():
        return 0
    _, h, d = t.shape
    st, sh, sd = t.stride()
    if sd == 1 and (sh == d or h == 1) and st >= h * d:     # a slice of a projection
        return st
    return binding._token_stride(name, t, 2)


def _attention_args(q, k_cache, v_cache, block_table, n, scale, window, sinks, max_new_len, splits):
    shape, dtype = q.shape, q.dtype
    if len(shape) != 3:
        _fail("q must be [T, Hq, D]")
    if dtype not in _DTYPES:
        _fail(f"unsupported dtype {dtype}", TypeError)
    T, hq, dim = shape
    if k_cache.dim() != 4:
        _fail("k_cache must be [pages, Hkv, page_size, D]")
    hkv = k_cache.shape[1]
    kp, vp, page_size, pages = _pools(k_cache, v_cache, dtype, hkv, dim)
    if hkv < 1 or hq % hkv != 0:
        _fail(f"Hq ({hq}) must be divisible by Hkv ({hkv})")
    stride, cols = _table(block_table, n)
    window, sinks = int(window), int(sinks)
    if window < 0 or sinks < 0:
        _fail("window and sinks must be >= 0")
    max_new_len, splits = int(max_new_len or 0), int(splits)
    if max_new_len < 0:
        _fail("max_new_len must be >= 0")
    if not 0 <= splits <= 64:
        _fail("splits must lie in [0, 64]")
    return PagedAttentionArgs(
        _SIZEOF_ATTENTION, None, None, None, None, None, None, None, None, None, 0, T,
        _rows_stride("q", q), kp, vp, stride, _DTYPES[dtype], n, hq, hkv, dim, page_size, pages, cols,
        min(window, 1 << 30), min(sinks, 1 << 30), min(max_new_len, 1 << 30), splits,
        float(dim ** -0.5 if scale is None else scale), None)


def _workspace_bytes(lib, a):
    nbytes = ctypes.c_size_t(0)
    st = lib.kda_paged_attention_workspace_size(ctypes.byref(a), ctypes.byref(nbytes))
    if st != KDA_OK:
        _raise(lib, st)
    return nbytes.value


def paged_attention_workspace_bytes(q, k_cache, v_cache, block_table, window=0, sinks=0,
                                    max_new_len=None, splits=0):
    """Workspace bytes that paged_attention needs for tensors of these shapes.  Smaller ones
    may be cut into more pieces and need more; PAGED_ATTENTION_WORKSPACE_MAX bytes serve
    every call.  The pieces follow the table's width: a step of short requests asks for
    less over the columns in use, block_table[:, :m]."""
    a = _attention_args(q, k_cache, v_cache, block_table, block_table.shape[0], None, window,
                        sinks, max_new_len, splits)
    return _workspace_bytes(load_library(), a)


def paged_attention(q, k_cache, v_cache, block_table, cu_seqlens, seq_lens, scale=None, window=0,
                    sinks=0, output=None, return_lse=False, lse=None, max_new_len=None,
                    workspace=None, splits=0):
    """Causal attention of each request's new tokens over its pages
    (kda_paged_attention); one new token per request is decode.

    q [T, Hq, D] bf16, fp16 or fp32 (D = 64 or 128; may be a view of a fused
    projection); k_cache, v_cache [pages, Hkv, page_size, D] of q's dtype, with the
    new tokens' rows already in them; block_table [n, max_pages] int32; cu_seqlens
    [n + 1]: request i's rows of q; seq_lens [n]: its cached keys, the new ones
    included.  window > 0 shows a row its last `window` keys (its own among them) and
    the request's first `sinks` ones.  A row that sees no key gets zeros; rows behind
    cu_seqlens[n] are left as they are (undefined where the output is allocated here).

    max_new_len: the longest request's new tokens, a planning hint (1 for decode; taken
    from cu_seqlens when that is a host tensor, unless a given workspace is too small for
    the plan that it leads to); results do not depend on it.
    splits: 0 lets the library cut long key ranges; else at most that many pieces.
    workspace: optional scratch of paged_attention_workspace_bytes() for these shapes, or
    of PAGED_ATTENTION_WORKSPACE_MAX for any, for one call at a time.  Returns out [T, Hq, D], or (out, lse [T, Hq] fp32) with return_lse."""
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        _fail("cu_seqlens must be [n + 1]")
    n = cu_seqlens.shape[0] - 1
    own_hint = max_new_len is None and n > 0 and cu_seqlens.device.type == "cpu"
    if own_hint:
        max_new_len = max(0, int((cu_seqlens[1:] - cu_seqlens[:-1]).max()))
    a = _attention_args(q, k_cache, v_cache, block_table, n, scale, window, sinks, max_new_len,
                        splits)
    dev = q.device
    cu = _int32(cu_seqlens, n + 1, "cu_seqlens", dev)
    seq = _int32(seq_lens, n, "seq_lens", dev)
    shape = q.shape
    if output is not None:
        _need(output.shape == shape, "output must have q's shape")
        _need(output.dtype is q.dtype, "output must have q's dtype", TypeError)
        _need(output.is_contiguous(), "output must be contiguous")
    if lse is not None:
        _need(lse.shape == shape[:2], "lse must be [T, Hq]")
        _need(lse.dtype is torch.float32, "lse must have dtype torch.float32", TypeError)
        _need(lse.is_contiguous(), "lse must be contiguous")
    if workspace is not None:
        _need(workspace.is_contiguous(), "workspace must be contiguous")
    _same_device(dev, k_cache=k_cache, v_cache=v_cache, block_table=block_table, output=output,
                 lse=lse, workspace=workspace)
    _on_gpu(dev)
    if output is None:
        output = torch.empty(shape, dtype=q.dtype, device=dev)
    if return_lse and lse is None:
        lse = torch.empty(shape[:2], dtype=torch.float32, device=dev)
    lib = _lib or load_library()
    if workspace is None:
        nbytes = _workspace_bytes(lib, a)
        if nbytes:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    elif own_hint and _workspace_bytes(lib, a) > workspace.numel() * workspace.element_size():
        a.max_new_len = 0       # its size was asked for without the offsets
    if workspace is not None:
        a.workspace = workspace.data_ptr()
        a.workspace_bytes = workspace.numel() * workspace.element_size()
    a.q, a.k_cache, a.v_cache = q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr()
    a.block_table, a.cu_seqlens, a.seq_lens = block_table.data_ptr(), cu.data_ptr(), seq.data_ptr()
    a.out, a.lse = output.data_ptr(), None if lse is None else lse.data_ptr()
    a.stream = _stream(dev)
    _call(lib.kda_paged_attention, a, dev)
    return (output, lse) if return_lse else output
