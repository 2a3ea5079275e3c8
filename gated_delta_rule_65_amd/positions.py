"""ctypes binding of the rotary positions (include/kda_rotary.h), and the frequencies
that they turn with.

``rotary`` turns a step's query and key rows to the positions that
``paged.page_tables`` gives, before ``paged.kv_append`` or ``paged_q8.kv_append_q8``
writes the keys.  As in ``binding``, this layer checks and marshals arguments only; the
rows are turned by the library's HIP kernel, queued on torch's current stream of their device.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import binding
from .binding import _DTYPES, _need
from .paged import _F, _I, _L, _P, _Z, _call, _fail, _on_gpu, _rows_stride, _stream


class RotaryArgs(ctypes.Structure):
    _fields_ = [
        ("struct_size", _Z),
        ("q", _P), ("k", _P), ("q_out", _P), ("k_out", _P),
        ("positions", _P), ("frequencies", _P),
        ("total_tokens", _L), ("q_stride", _L), ("k_stride", _L),
        ("q_out_stride", _L), ("k_out_stride", _L),
        ("dtype", _I), ("hq", _I), ("hk", _I), ("head_dim", _I), ("pairs", _I),
        ("interleaved", _I), ("inverse", _I), ("scale", _F), ("stream", _P),
    ]


_SIZEOF = ctypes.sizeof(RotaryArgs)
_INT32, _FP64, _DENSE = torch.int32, torch.float64, torch.contiguous_format
EXPORTS = ("kda_rotary",)
_lib = None


def load_library():
    """The library with the rotary entry point declared; raises if it is missing."""
    global _lib
    if _lib is None:
        lib = binding.load_library()
        lib.kda_rotary.argtypes, lib.kda_rotary.restype = [ctypes.POINTER(RotaryArgs)], ctypes.c_int
        _lib = lib
    return _lib


def rotary_frequencies(rotary_dim, base=10000.0, scaling=None, factor=1.0, original_length=None,
                       slow_turns=1.0, fast_turns=32.0, device=None):
    """Radians per position of the pairs of `rotary_dim` channels: [rotary_dim / 2] fp64,
    base^(-2 i / rotary_dim), computed once and kept by the caller.

    scaling: how a context `factor` times as long as the trained one is fitted in.
      None      not at all
      "linear"  every frequency divided by factor
      "base"    base times factor^(d / (d - 2)), d = rotary_dim: the fastest pair keeps its
                frequency, the slowest one is divided by factor
      "turns"   pairs that make fast_turns turns and more over original_length positions keep theirs,
                those of slow_turns and fewer are divided by factor, with a ramp over the
                pair index between, its ends rounded outward to whole pairs from the first one
                on (the `scale` of rotary is then usually 0.1 ln(factor) + 1)
    """
    rotary_dim = int(rotary_dim)
    if rotary_dim < 2 or rotary_dim % 2:
        _fail("rotary_dim must be even and >= 2")
    if not (math.isfinite(base) and base > 0):
        _fail("base must be above 0 and finite")
    if not (math.isfinite(factor) and factor > 0):
        _fail("factor must be above 0 and finite")
    i = torch.arange(rotary_dim // 2, dtype=torch.float64)
    if scaling == "base":
        if rotary_dim == 2:
            _fail('scaling "base" needs more than one pair')
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f = torch.pow(torch.tensor(float(base), dtype=torch.float64), -2 * i / rotary_dim)
    if scaling == "linear":
        f = f / factor
    elif scaling == "turns":
        if original_length is None or not original_length > 0:
            _fail('scaling "turns" needs original_length > 0')
        if not (0 < slow_turns < fast_turns):
            _fail("turns must satisfy 0 < slow_turns < fast_turns")
        if base <= 1.0:
            _fail('scaling "turns" needs a base above 1')

        def index(turns):       # of the pair that makes this many turns
            return rotary_dim * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))

        lo = max(math.floor(index(fast_turns)), 0)
        hi = max(math.ceil(index(slow_turns)), 0)
        slow = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = f * (1 - slow) + f / factor * slow
    elif scaling not in (None, "base"):
        _fail(f"unknown scaling {scaling!r}")
    return f if device is None else f.to(device)


def rotary(q, k, positions, frequencies, interleaved=False, scale=1.0, inverse=False, q_out=None,
           k_out=None):
    """Turns the rows of q [T, Hq, D] and k [T, Hk, D] (or None) to their positions
    (kda_rotary); returns (q_out, k_out).

    positions [T] int32: rows at a negative one (behind a step's last token, as
    page_tables marks them) are not written, so undefined where the output is allocated here.
    frequencies [n] fp64 on the rows' device (rotary_frequencies): pair i of the first
    2 n channels is (i, i + n), or (2 i, 2 i + 1) with interleaved, and turns by
    positions * frequencies[i]; the result is times scale, and other channels pass unchanged.
    inverse turns back, with the same scale: the gradient with respect to q and k, given that
    with respect to the outputs in their place.  bf16, fp16 or fp32, D a multiple of 8 up to
    512; q and k may be views of a fused projection.  q_out and k_out may be q and k themselves (in
    place) and otherwise share no memory with them."""
    if q.dim() != 3:
        _fail("q must be [T, Hq, D]")
    T, hq, dim = q.shape
    dtype = q.dtype
    code = _DTYPES.get(dtype)
    if code is None:
        _fail(f"unsupported dtype {dtype}", TypeError)
    if positions.shape != (T,):
        _fail(f"positions must have shape [{T}]")
    if positions.dtype is not _INT32:
        _fail("positions must have dtype torch.int32", TypeError)
    if frequencies.dim() != 1:
        _fail("frequencies must be [n]")
    n = frequencies.shape[0]
    if not 1 <= n <= dim // 2:
        _fail(f"frequencies must be [n] with 1 <= n <= {dim // 2}")
    if frequencies.dtype is not _FP64:
        _fail("frequencies must have dtype torch.float64", TypeError)
    if not (positions.is_contiguous() and frequencies.is_contiguous()):
        _fail("positions and frequencies must be contiguous")
    on = q.get_device()
    if positions.get_device() != on or frequencies.get_device() != on:
        _fail(f"positions and frequencies must be on {q.device}")
    qs = _rows_stride("q", q)
    ks = kos = hk = 0
    if k is None:
        if k_out is not None:
            _fail("k_out without k")
    else:
        if k.dim() != 3 or k.shape[0] != T or k.shape[2] != dim:
            _fail(f"k must be [{T}, Hk, {dim}]")
        if k.dtype is not dtype:
            _fail(f"k must have dtype {dtype}", TypeError)
        if k.get_device() != on:
            _fail(f"k must be on {q.device}")
        hk = k.shape[1]
        ks = _rows_stride("k", k)
        if k_out is not None:
            kos = _out_stride("k", k, k_out, ks)
    qos = 0 if q_out is None else _out_stride("q", q, q_out, qs)
    dev = q.device
    _on_gpu(dev)
    if q_out is None:
        q_out = torch.empty_like(q, memory_format=_DENSE)
    if k is None:
        k_at = k_out_at = None
    else:
        if k_out is None:
            k_out = torch.empty_like(k, memory_format=_DENSE)
        k_at, k_out_at = k.data_ptr(), k_out.data_ptr()
    lib = _lib or load_library()
    _call(lib.kda_rotary, RotaryArgs(
        _SIZEOF, q.data_ptr(), k_at, q_out.data_ptr(), k_out_at, positions.data_ptr(),
        frequencies.data_ptr(), T, qs, ks, qos, kos, code, hq, hk, dim, n, bool(interleaved),
        bool(inverse), float(scale), _stream(dev)), dev)
    return q_out, k_out


def _out_stride(name, x, out, stride):
    """Elements between the tokens of the rows that x is turned into."""
    if out is x:
        return stride
    _need(out.shape == x.shape, f"{name}_out must have {name}'s shape")
    _need(out.dtype is x.dtype, f"{name}_out must have {name}'s dtype", TypeError)
    _need(out.device == x.device, f"{name}_out must be on {x.device}")
    return _rows_stride(name + "_out", out)
