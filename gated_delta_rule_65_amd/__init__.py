"""MI355X-native KDA (Kimi Delta Attention) chunked forward and paged decode,
with the paged softmax attention of the layers that stand between KDA layers: rotary
positions, and a cache in 16 or 8 bits.

The compute lives in a C-ABI shared library of hand-written gfx950 HIP
kernels (``csrc/``, declared in ``include/kda.h``, ``kda_paged.h``, ``kda_paged_q8.h``
and ``kda_rotary.h``); ``binding``, ``paged``, ``paged_q8`` and ``positions`` are thin
ctypes layers over it.  Importing the package
does not load the library; the first call does, and raises if it is missing.
"""
_EXPORTS = ("KdaError", "chunk_kda", "kda_decode", "chunk_stages", "library_path",
            "load_library")
_PAGED = ("PageTables", "page_tables", "kv_append", "paged_attention",
          "paged_attention_workspace_bytes", "PAGED_ATTENTION_WORKSPACE_MAX")

_PAGED_Q8 = ("kv_append_q8", "kv_read_q8", "paged_attention_q8",
             "paged_attention_q8_workspace_bytes")
_POSITIONS = ("rotary", "rotary_frequencies")


def __getattr__(name):
    if name in _POSITIONS:
        from . import positions
        return getattr(positions, name)
    if name in _PAGED_Q8:
        from . import paged_q8
        return getattr(paged_q8, name)
    if name in _PAGED:
        from . import paged
        return getattr(paged, name)
    if name in _EXPORTS:
        from . import binding
        return getattr(binding, name)
    raise AttributeError(name)


__all__ = list(_EXPORTS + _PAGED + _PAGED_Q8 + _POSITIONS)
