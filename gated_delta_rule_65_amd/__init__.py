"""MI355X-native KDA (Kimi Delta Attention) chunked forward and paged decode,
with the paged softmax attention of the layers that stand between KDA layers.

The compute lives in a C-ABI shared library of hand-written gfx950 HIP
kernels (``csrc/``, declared in ``include/kda.h`` and ``include/kda_paged.h``);
``binding`` and ``paged`` are thin ctypes layers over it.  Importing the package
does not load the library; the first call does, and raises if it is missing.
"""
_EXPORTS = ("KdaError", "chunk_kda", "kda_decode", "chunk_stages", "library_path",
            "load_library")
_PAGED = ("PageTables", "page_tables", "kv_append", "paged_attention",
          "paged_attention_workspace_bytes", "PAGED_ATTENTION_WORKSPACE_MAX")


def __getattr__(name):
    if name in _PAGED:
        from . import paged
        return getattr(paged, name)
    if name in _EXPORTS:
        from . import binding
        return getattr(binding, name)
    raise AttributeError(name)


__all__ = list(_EXPORTS + _PAGED)
