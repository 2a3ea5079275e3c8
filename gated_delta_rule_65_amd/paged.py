"""ctypes binding of the paged attention operators (include/kda_paged.h).

The attention side of a hybrid model's serving step, beside the KDA layers of
``binding``: the step's block tables and slot maps (``page_tables``), the new key
and value rows into the paged cache (``kv_append``) and the attention over it
(``paged_attention``).  As in ``binding``, this layer checks and marshals arguments
only; every step of the computation runs in the library's HIP kernels, queued on
torch's current stream of the tensors' device.
"""
from __future__ import annotations

import contextlib
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


EXPORTS = ("kda_page_tables", "kda_kv_append", "kda_paged_attention_workspace_size",
           "kda_paged_attention")
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


def _on_gpu(dev):
    _need(dev.type == "cuda", f"tensors must be on a GPU, got {dev}")


def _same_device(dev, **tensors):
    for name, t in tensors.items():
        _need(t is None or t.device == dev, f"{name} must be on {dev}")


def _guard(dev):
    """Makes the tensors' device current for the launch."""
    if dev.index is None or dev.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(dev)


def _int32(x, shape, name, dev):
    _need(tuple(x.shape) == shape, f"{name} must have shape {list(shape)}")
    if x.dtype != torch.int32:
        _need(x.dtype == torch.int64, f"{name} must have dtype torch.int32 or torch.int64",
              TypeError)
    return x.to(device=dev, dtype=torch.int32).contiguous()


def _table(block_table, n):
    """(row stride, columns) of an int32 [n, max_pages] block table."""
    _need(block_table.dim() == 2 and block_table.shape[0] == n,
          f"block_table must be [{n}, max_pages]")
    _need(block_table.dtype == torch.int32, "block_table must have dtype torch.int32", TypeError)
    cols = block_table.shape[1]
    if block_table.is_contiguous():
        return cols, cols
    _need((cols == 1 or block_table.stride(1) == 1) and
          (n == 1 or block_table.stride(0) >= cols), "block_table rows must be dense")
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
    _need(k_cache.dim() == 4 and k_cache.shape[1] == hkv and k_cache.shape[3] == dim,
          f"k_cache must be [pages, {hkv}, page_size, {dim}]")
    _need(v_cache.shape == k_cache.shape, "v_cache must have k_cache's shape")
    _need(k_cache.dtype == dtype and v_cache.dtype == dtype,
          f"k_cache and v_cache must have dtype {dtype}", TypeError)
    return _page_stride("k_cache", k_cache), _page_stride("v_cache", v_cache)


def page_tables(context_lens, new_lens, free_pages, block_table, page_size, num_pages,
                max_tokens=None, out=None):
    """A step's block tables and slot maps, built on the GPU from the requests'
    lengths (kda_page_tables).

    context_lens, new_lens [n]: cached and new tokens per request; free_pages [F]:
    page ids to take from, in order; block_table [n, max_pages] int32, updated in
    place (the entries of the pages taken; rows may lie apart); num_pages: pages of
    the cache.  max_tokens: room in the slot map, at least the step's new tokens (a
    captured step keeps its largest).  Returns a PageTables; ``out`` gives one to
    write into (its slot_mapping then sets max_tokens)."""
    n = context_lens.shape[0] if context_lens.dim() == 1 else -1
    _need(n >= 0, "context_lens must be [n]")
    _need(free_pages.dim() == 1, "free_pages must be [F]")
    stride, cols = _table(block_table, n)
    _need(int(page_size) >= 1, "page_size must be >= 1")
    dev = block_table.device
    ctx = _int32(context_lens, (n,), "context_lens", dev)
    new = _int32(new_lens, (n,), "new_lens", dev)
    free = _int32(free_pages, (free_pages.shape[0],), "free_pages", dev)
    if out is None:
        _need(max_tokens is not None and int(max_tokens) >= 0,
              "max_tokens is needed (the room for new tokens)")
        tokens = int(max_tokens)
        ints = torch.empty(2 * n + 2 + tokens, dtype=torch.int32, device=dev)
        cu, seq, taken, pos = torch.split(ints, [n + 1, n, 1, tokens])
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
            _need(tuple(t.shape) == shape, f"out.{name} must have shape {list(shape)}")
            _need(t.dtype == dt, f"out.{name} must have dtype {dt}", TypeError)
            _need(t.is_contiguous(), f"out.{name} must be contiguous")
            _need(t.device == dev, f"out.{name} must be on {dev}")
    _on_gpu(dev)
    lib = load_library()
    with _guard(dev):
        a = PageTablesArgs(
            ctypes.sizeof(PageTablesArgs), ctx.data_ptr(), new.data_ptr(), free.data_ptr(),
            block_table.data_ptr(), stride, n, free.shape[0], cols, int(page_size),
            int(num_pages), tokens, out.slot_mapping.data_ptr(), out.positions.data_ptr(),
            out.cu_seqlens.data_ptr(), out.seq_lens.data_ptr(), out.pages_taken.data_ptr(),
            torch.cuda.current_stream(dev).cuda_stream)
        st = lib.kda_page_tables(ctypes.byref(a))
    if st != KDA_OK:
        _raise(lib, st)
    return out


def kv_append(k, v, k_cache, v_cache, slot_mapping):
    """Copies the rows k, v [T, Hkv, D] to their slots of the paged caches
    [pages, Hkv, page_size, D], in place (kda_kv_append).  slot_mapping [T] int64
    holds distinct slots page * page_size + offset; one outside the cache (-1) skips
    its token.  k and v may be views of a fused projection."""
    _need(k.dim() == 3, "k must be [T, Hkv, D]")
    _need(v.shape == k.shape, "v must have k's shape")
    _need(k.dtype in _DTYPES, f"unsupported dtype {k.dtype}", TypeError)
    _need(v.dtype == k.dtype, "v must have k's dtype", TypeError)
    T, hkv, dim = k.shape
    kp, vp = _pools(k_cache, v_cache, k.dtype, hkv, dim)
    _need(slot_mapping.dim() == 1 and slot_mapping.shape[0] == T, f"slot_mapping must have shape [{T}]")
    _need(slot_mapping.dtype == torch.int64, "slot_mapping must have dtype torch.int64", TypeError)
    _need(slot_mapping.is_contiguous(), "slot_mapping must be contiguous")
    ks, vs = binding._token_stride("k", k, 2), binding._token_stride("v", v, 2)
    dev = k.device
    _same_device(dev, v=v, k_cache=k_cache, v_cache=v_cache, slot_mapping=slot_mapping)
    _on_gpu(dev)
    lib = load_library()
    with _guard(dev):
        a = KvAppendArgs(
            ctypes.sizeof(KvAppendArgs), k.data_ptr(), v.data_ptr(), k_cache.data_ptr(),
            v_cache.data_ptr(), slot_mapping.data_ptr(), T, ks, vs, kp, vp, _DTYPES[k.dtype], hkv,
            dim, k_cache.shape[2], k_cache.shape[0], torch.cuda.current_stream(dev).cuda_stream)
        st = lib.kda_kv_append(ctypes.byref(a))
    if st != KDA_OK:
        _raise(lib, st)


def _attention_args(q, k_cache, v_cache, block_table, n, scale, window, sinks, max_new_len, splits):
    _need(q.dim() == 3, "q must be [T, Hq, D]")
    _need(q.dtype in _DTYPES, f"unsupported dtype {q.dtype}", TypeError)
    T, hq, dim = q.shape
    _need(k_cache.dim() == 4, "k_cache must be [pages, Hkv, page_size, D]")
    hkv = k_cache.shape[1]
    kp, vp = _pools(k_cache, v_cache, q.dtype, hkv, dim)
    _need(hkv > 0 and hq % hkv == 0, f"Hq ({hq}) must be divisible by Hkv ({hkv})")
    stride, cols = _table(block_table, n)
    _need(int(window) >= 0 and int(sinks) >= 0, "window and sinks must be >= 0")
    return PagedAttentionArgs(
        ctypes.sizeof(PagedAttentionArgs), None, None, None, None, None, None, None, None, None, 0,
        T, binding._token_stride("q", q, 2), kp, vp, stride, _DTYPES[q.dtype], n, hq, hkv, dim,
        k_cache.shape[2], k_cache.shape[0], cols, min(int(window), 1 << 30),
        min(int(sinks), 1 << 30), int(max_new_len or 0), int(splits),
        float(dim ** -0.5 if scale is None else scale), None)


def paged_attention_workspace_bytes(q, k_cache, v_cache, block_table, window=0, sinks=0,
                                    max_new_len=None, splits=0):
    """Workspace bytes that paged_attention needs for tensors of these shapes."""
    a = _attention_args(q, k_cache, v_cache, block_table, block_table.shape[0], None, window,
                        sinks, max_new_len, splits)
    lib = load_library()
    nbytes = ctypes.c_size_t(0)
    st = lib.kda_paged_attention_workspace_size(ctypes.byref(a), ctypes.byref(nbytes))
    if st != KDA_OK:
        _raise(lib, st)
    return int(nbytes.value)


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

    max_new_len: the longest request's new tokens, a planning hint (1 for decode).
    splits: 0 lets the library cut long key ranges; else at most that many pieces.
    workspace: optional scratch of paged_attention_workspace_bytes(), for one call at
    a time.  Returns out [T, Hq, D], or (out, lse [T, Hq] fp32) with return_lse."""
    n = cu_seqlens.shape[0] - 1 if cu_seqlens.dim() == 1 else -1
    _need(n >= 0, "cu_seqlens must be [n + 1]")
    a = _attention_args(q, k_cache, v_cache, block_table, n, scale, window, sinks, max_new_len,
                        splits)
    dev = q.device
    cu = _int32(cu_seqlens, (n + 1,), "cu_seqlens", dev)
    seq = _int32(seq_lens, (n,), "seq_lens", dev)
    shape = tuple(q.shape)
    if output is not None:
        _need(tuple(output.shape) == shape, "output must have q's shape")
        _need(output.dtype == q.dtype, "output must have q's dtype", TypeError)
        _need(output.is_contiguous(), "output must be contiguous")
    if lse is not None:
        _need(tuple(lse.shape) == shape[:2], "lse must be [T, Hq]")
        _need(lse.dtype == torch.float32, "lse must have dtype torch.float32", TypeError)
        _need(lse.is_contiguous(), "lse must be contiguous")
    _same_device(dev, k_cache=k_cache, v_cache=v_cache, block_table=block_table, output=output,
                 lse=lse, workspace=workspace)
    _on_gpu(dev)
    if output is None:
        output = torch.empty(shape, dtype=q.dtype, device=dev)
    if return_lse and lse is None:
        lse = torch.empty(shape[:2], dtype=torch.float32, device=dev)
    lib = load_library()
    with _guard(dev):
        nbytes = ctypes.c_size_t(0)
        st = lib.kda_paged_attention_workspace_size(ctypes.byref(a), ctypes.byref(nbytes))
        if st != KDA_OK:
            _raise(lib, st)
        if workspace is None and nbytes.value:
            workspace = torch.empty(nbytes.value, dtype=torch.uint8, device=dev)
        if workspace is not None:
            _need(workspace.is_contiguous(), "workspace must be contiguous")
            a.workspace = workspace.data_ptr()
            a.workspace_bytes = workspace.numel() * workspace.element_size()
        a.q, a.k_cache, a.v_cache = q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr()
        a.block_table, a.cu_seqlens, a.seq_lens = block_table.data_ptr(), cu.data_ptr(), seq.data_ptr()
        a.out, a.lse = output.data_ptr(), None if lse is None else lse.data_ptr()
        a.stream = torch.cuda.current_stream(dev).cuda_stream
        st = lib.kda_paged_attention(ctypes.byref(a))
    if st != KDA_OK:
        _raise(lib, st)
    return (output, lse) if return_lse else output
