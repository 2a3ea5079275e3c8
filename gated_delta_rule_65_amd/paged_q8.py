"""ctypes binding of the paged cache in 8 bits (include/kda_paged_q8.h).

The operators of ``paged`` over a cache of half the bytes: codes (e4m3 or int8) with a
power-of-two scale per block of positions and head.  A step's new rows go in with
``kv_append_q8``, ``paged_attention_q8`` attends over them, and ``kv_read_q8`` gives cached rows back.
All three address rows by the tables of ``paged.page_tables``.  As in ``binding``, this
layer checks and marshals arguments only; every step of the computation runs in the
library's HIP kernels, queued on torch's current stream of the tensors' device.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding
from .binding import KDA_OK, _DTYPES, _need, _raise
from .paged import (_F, _I, _L, _P, _Z, _call, _fail, _int32, _on_gpu, _page_stride, _rows_stride,
                    _same_device, _stream, _table)

_CODES = {torch.float8_e4m3fn: 0, torch.int8: 1}
_FP32, _BF16, _FP16 = torch.float32, torch.bfloat16, torch.float16
_DENSE = torch.contiguous_format


class KvAppendQ8Args(ctypes.Structure):
    _fields_ = [
        ("struct_size", _Z),
        ("k", _P), ("v", _P), ("k_cache", _P), ("v_cache", _P), ("k_scale", _P), ("v_scale", _P),
        ("block_table", _P), ("cu_seqlens", _P), ("seq_lens", _P),
        ("total_tokens", _L), ("k_stride", _L), ("v_stride", _L),
        ("k_page_stride", _L), ("v_page_stride", _L), ("table_stride", _L),
        ("dtype", _I), ("code", _I), ("n", _I), ("hkv", _I), ("head_dim", _I), ("page_size", _I),
        ("block", _I), ("num_pages", _I), ("max_pages", _I), ("stream", _P),
    ]


class KvReadQ8Args(ctypes.Structure):
    _fields_ = [
        ("struct_size", _Z),
        ("k_cache", _P), ("v_cache", _P), ("k_scale", _P), ("v_scale", _P),
        ("block_table", _P), ("cu_seqlens", _P), ("seq_lens", _P), ("k_out", _P), ("v_out", _P),
        ("total_tokens", _L), ("k_page_stride", _L), ("v_page_stride", _L), ("table_stride", _L),
        ("dtype", _I), ("code", _I), ("n", _I), ("hkv", _I), ("head_dim", _I), ("page_size", _I),
        ("block", _I), ("num_pages", _I), ("max_pages", _I), ("stream", _P),
    ]


class PagedAttentionQ8Args(ctypes.Structure):
    _fields_ = [
        ("struct_size", _Z),
        ("q", _P), ("k_cache", _P), ("v_cache", _P), ("k_scale", _P), ("v_scale", _P),
        ("block_table", _P), ("cu_seqlens", _P),
        ("seq_lens", _P), ("out", _P), ("lse", _P), ("workspace", _P), ("workspace_bytes", _Z),
        ("total_tokens", _L), ("q_stride", _L), ("k_page_stride", _L), ("v_page_stride", _L),
        ("table_stride", _L),
        ("dtype", _I), ("code", _I), ("n", _I), ("hq", _I), ("hkv", _I),
        ("head_dim", _I), ("page_size", _I), ("block", _I), ("num_pages", _I), ("max_pages", _I),
        ("window", _I), ("sinks", _I), ("max_new_len", _I), ("splits", _I),
        ("scale", _F), ("stream", _P),
    ]


_SIZEOF_APPEND = ctypes.sizeof(KvAppendQ8Args)
_SIZEOF_READ = ctypes.sizeof(KvReadQ8Args)
_SIZEOF_ATTENTION = ctypes.sizeof(PagedAttentionQ8Args)

EXPORTS = ("kda_kv_append_q8", "kda_kv_read_q8", "kda_paged_attention_q8_workspace_size",
           "kda_paged_attention_q8")
_lib = None


def load_library():
    """The library with the entry points of the 8-bit cache declared; raises if it is missing."""
    global _lib
    if _lib is None:
        lib = binding.load_library()
        P = ctypes.POINTER
        for name, args in (("kda_kv_append_q8", [P(KvAppendQ8Args)]),
                           ("kda_kv_read_q8", [P(KvReadQ8Args)]),
                           ("kda_paged_attention_q8", [P(PagedAttentionQ8Args)]),
                           ("kda_paged_attention_q8_workspace_size",
                            [P(PagedAttentionQ8Args), P(ctypes.c_size_t)])):
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, ctypes.c_int
        _lib = lib
    return _lib


def _codes(k_cache, v_cache, k_scale, v_scale):
    """(code, K page stride, V page stride, pages, Hkv, page size, D, block) of a cache."""
    shape, dtype = k_cache.shape, k_cache.dtype
    if len(shape) != 4:
        _fail("k_cache must be [pages, Hkv, page_size, D]")
    if v_cache.shape != shape:
        _fail("v_cache must have k_cache's shape")
    code = _CODES.get(dtype)
    if code is None:
        _fail(f"k_cache must have dtype torch.float8_e4m3fn or torch.int8, got {dtype}", TypeError)
    if v_cache.dtype is not dtype:
        _fail("v_cache must have k_cache's dtype", TypeError)
    pages, hkv, page_size, dim = shape
    ss = k_scale.shape
    blocks = ss[2] if len(ss) == 3 and ss[0] == pages and ss[1] == hkv else 0
    if blocks < 1 or page_size % blocks:
        _fail(f"k_scale must be [{pages}, {hkv}, blocks], blocks a divisor of page_size ({page_size})")
    if v_scale.shape != ss:
        _fail("v_scale must have k_scale's shape")
    if k_scale.dtype is not _FP32 or v_scale.dtype is not _FP32:
        _fail("k_scale and v_scale must have dtype torch.float32", TypeError)
    if not (k_scale.is_contiguous() and v_scale.is_contiguous()):
        _fail("k_scale and v_scale must be contiguous")
    return (code, _page_stride("k_cache", k_cache), _page_stride("v_cache", v_cache), pages, hkv,
            page_size, dim, page_size // blocks)


def _cache_device(on, k_cache, v_cache, k_scale, v_scale, block_table):
    """Whether a cache and its table are on the device of this index (-1 the host's); indexes cost
    less than devices."""
    return (k_cache.get_device() == on and v_cache.get_device() == on and k_scale.get_device() == on
            and v_scale.get_device() == on and block_table.get_device() == on)


def _requests(block_table, cu_seqlens, seq_lens, dev):
    """(requests, offsets, lengths, table stride, columns)."""
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        _fail("cu_seqlens must be [n + 1]")
    n = cu_seqlens.shape[0] - 1
    stride, cols = _table(block_table, n)
    return (n, _int32(cu_seqlens, n + 1, "cu_seqlens", dev), _int32(seq_lens, n, "seq_lens", dev),
            stride, cols)


def kv_append_q8(k, v, k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens, seq_lens):
    """Writes the rows k, v [T, Hkv, D] of a step to their places in the cache in 8 bits,
    in place (kda_kv_append_q8).

    k_cache, v_cache [pages, Hkv, page_size, D] float8_e4m3fn or int8; k_scale, v_scale
    [pages, Hkv, blocks] fp32, a scale per page_size / blocks positions; block_table
    [n, max_pages] int32, cu_seqlens [n + 1], seq_lens [n] as paged_attention takes them: request i's rows are its
    newest positions, seq_lens its cached positions with these.  A row without a page is skipped.

    A block's scale is the least power of two with which its rows are codes; rows that
    join earlier ones keep the scale or raise it, and the earlier codes are then rounded to it.
    The scales of blocks that have no rows yet need no initial value.  Scales written elsewhere have to be
    powers of two too: any other counts as the next one below, here and in every reader.  k and v (bf16, fp16 or fp32)
    may be views of a fused projection."""
    shape, dtype = k.shape, k.dtype
    if len(shape) != 3:
        _fail("k must be [T, Hkv, D]")
    if v.shape != shape:
        _fail("v must have k's shape")
    if dtype not in _DTYPES:
        _fail(f"unsupported dtype {dtype}", TypeError)
    if v.dtype is not dtype:
        _fail("v must have k's dtype", TypeError)
    code, kp, vp, pages, hkv, page_size, dim, block = _codes(k_cache, v_cache, k_scale, v_scale)
    if shape[1] != hkv or shape[2] != dim:
        _fail(f"k must be [T, {hkv}, {dim}]")
    dev = k.device
    n, cu, seq, stride, cols = _requests(block_table, cu_seqlens, seq_lens, dev)
    ks, vs = _rows_stride("k", k), _rows_stride("v", v)
    on = k.get_device()
    if v.get_device() != on or not _cache_device(on, k_cache, v_cache, k_scale, v_scale, block_table):
        _same_device(dev, v=v, k_cache=k_cache, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale,
                     block_table=block_table)
    _on_gpu(dev)
    lib = _lib or load_library()
    _call(lib.kda_kv_append_q8, KvAppendQ8Args(
        _SIZEOF_APPEND, k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(), cu.data_ptr(), seq.data_ptr(),
        shape[0], ks, vs, kp, vp, stride, _DTYPES[dtype], code, n, hkv, dim, page_size, block, pages, cols,
        _stream(dev)), dev)


def kv_read_q8(k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens, seq_lens,
               total_tokens=None, dtype=torch.bfloat16, k_out=None, v_out=None):
    """The values of the requests' newest positions, (k, v) [T, Hkv, D] rounded to dtype
    (kda_kv_read_q8): request i's rows cu_seqlens[i] .. cu_seqlens[i + 1] are its positions up to
    seq_lens[i].  cu_seqlens of the running sums of seq_lens reads whole contexts.

    A row without a page gives zeros; rows behind cu_seqlens[n] are left as they are
    (undefined where the output is allocated here).  T is total_tokens, or the rows of k_out and
    v_out, or the last offset where cu_seqlens is a host tensor."""
    code, kp, vp, pages, hkv, page_size, dim, block = _codes(k_cache, v_cache, k_scale, v_scale)
    dev = k_cache.device
    if (k_out is None) != (v_out is None):
        _fail("k_out and v_out go together")
    if k_out is not None:
        dtype = k_out.dtype
        if total_tokens is None:
            total_tokens = k_out.shape[0]
    if dtype not in _DTYPES:
        _fail(f"unsupported dtype {dtype}", TypeError)
    if total_tokens is None:
        if cu_seqlens.device.type != "cpu" or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
            _fail("total_tokens is needed where cu_seqlens is on the GPU")
        total_tokens = int(cu_seqlens[-1])
    total_tokens = int(total_tokens)
    if total_tokens < 0:
        _fail("total_tokens must be >= 0")
    n, cu, seq, stride, cols = _requests(block_table, cu_seqlens, seq_lens, dev)
    shape = (total_tokens, hkv, dim)
    if k_out is not None:
        for name, t in (("k_out", k_out), ("v_out", v_out)):
            _need(t.shape == shape, f"{name} must have shape {list(shape)}")
            _need(t.dtype is dtype, f"{name} must have k_out's dtype", TypeError)
            _need(t.is_contiguous(), f"{name} must be contiguous")
        _same_device(dev, k_out=k_out, v_out=v_out)
    if not _cache_device(k_cache.get_device(), k_cache, v_cache, k_scale, v_scale, block_table):
        _same_device(dev, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale, block_table=block_table)
    _on_gpu(dev)
    if k_out is None:
        k_out = torch.empty(shape, dtype=dtype, device=dev)
        v_out = torch.empty_like(k_out)
    lib = _lib or load_library()
    _call(lib.kda_kv_read_q8, KvReadQ8Args(
        _SIZEOF_READ, k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
        block_table.data_ptr(), cu.data_ptr(), seq.data_ptr(), k_out.data_ptr(), v_out.data_ptr(),
        total_tokens, kp, vp, stride, _DTYPES[dtype], code, n, hkv, dim, page_size, block, pages, cols,
        _stream(dev)), dev)
    return k_out, v_out


def _attention_args(q, k_cache, v_cache, k_scale, v_scale, block_table, n, scale, window, sinks,
                    max_new_len, splits):
    shape, dtype = q.shape, q.dtype
    if len(shape) != 3:
        _fail("q must be [T, Hq, D]")
    if dtype is not _BF16 and dtype is not _FP16:
        _fail(f"q must have dtype torch.bfloat16 or torch.float16, got {dtype}", TypeError)
    T, hq, dim = shape
    code, kp, vp, pages, hkv, page_size, kdim, block = _codes(k_cache, v_cache, k_scale, v_scale)
    if kdim != dim:
        _fail(f"k_cache must be [pages, Hkv, page_size, {dim}]")
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
    return PagedAttentionQ8Args(
        _SIZEOF_ATTENTION, None, None, None, None, None, None, None, None, None, None, None, 0, T,
        _rows_stride("q", q), kp, vp, stride, _DTYPES[dtype], code, n, hq, hkv, dim, page_size, block,
        pages, cols, min(window, 1 << 30), min(sinks, 1 << 30), min(max_new_len, 1 << 30), splits,
        float(dim ** -0.5 if scale is None else scale), None)


def _workspace_bytes(lib, a):
    nbytes = ctypes.c_size_t(0)
    st = lib.kda_paged_attention_q8_workspace_size(ctypes.byref(a), ctypes.byref(nbytes))
    if st != KDA_OK:
        _raise(lib, st)
    return nbytes.value


def paged_attention_q8_workspace_bytes(q, k_cache, v_cache, k_scale, v_scale, block_table, window=0,
                                       sinks=0, max_new_len=None, splits=0):
    """Workspace bytes that paged_attention_q8 needs for tensors of these shapes, as
    paged_attention_workspace_bytes; PAGED_ATTENTION_WORKSPACE_MAX bytes serve every call."""
    a = _attention_args(q, k_cache, v_cache, k_scale, v_scale, block_table, block_table.shape[0], None,
                        window, sinks, max_new_len, splits)
    return _workspace_bytes(load_library(), a)


def paged_attention_q8(q, k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens, seq_lens,
                       scale=None, window=0, sinks=0, output=None, return_lse=False, lse=None,
                       max_new_len=None, workspace=None, splits=0):
    """paged_attention over a cache in 8 bits (kda_paged_attention_q8): causal attention of each request's
    new tokens over its pages; one new token per request is decode.

    q [T, Hq, D] bf16 or fp16 (D = 64 or 128; may be a view of a fused projection); the cache as
    kv_append_q8 takes it, with the new tokens' rows already in it.  Everything else is
    paged_attention's: block_table, cu_seqlens, seq_lens, window, sinks, max_new_len, workspace
    (of paged_attention_q8_workspace_bytes() or PAGED_ATTENTION_WORKSPACE_MAX bytes), splits.
    Returns out [T, Hq, D], or (out, lse [T, Hq] fp32) with return_lse."""
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        _fail("cu_seqlens must be [n + 1]")
    n = cu_seqlens.shape[0] - 1
    own_hint = max_new_len is None and n > 0 and cu_seqlens.device.type == "cpu"
    if own_hint:
        max_new_len = max(0, int((cu_seqlens[1:] - cu_seqlens[:-1]).max()))
    a = _attention_args(q, k_cache, v_cache, k_scale, v_scale, block_table, n, scale, window, sinks,
                        max_new_len, splits)
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
    if not _cache_device(q.get_device(), k_cache, v_cache, k_scale, v_scale, block_table):
        _same_device(dev, k_cache=k_cache, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale,
                     block_table=block_table)
    if not (output is None and lse is None and workspace is None):
        _same_device(dev, output=output, lse=lse, workspace=workspace)
    _on_gpu(dev)
    if output is None:
        output = torch.empty_like(q, memory_format=_DENSE)
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
    a.k_scale, a.v_scale = k_scale.data_ptr(), v_scale.data_ptr()
    a.block_table, a.cu_seqlens, a.seq_lens = block_table.data_ptr(), cu.data_ptr(), seq.data_ptr()
    a.out, a.lse = output.data_ptr(), None if lse is None else lse.data_ptr()
    a.stream = _stream(dev)
    _call(lib.kda_paged_attention_q8, a, dev)
    return (output, lse) if return_lse else output
