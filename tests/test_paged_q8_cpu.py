"""The C ABI and binding of the paged cache in 8 bits on the host: exports, struct agreement,
argument checks and launch plans.  No call here gets as far as queueing work."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import q8_ref as Q
from gated_delta_rule_65_amd import binding as B
from gated_delta_rule_65_amd import paged as P
from gated_delta_rule_65_amd import paged_q8 as P8

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20      # a well-aligned address that no check reads through
ARG, SHAPE, DTYPE, UNSUP, WS = (B.KDA_ERR_ARG, B.KDA_ERR_SHAPE, B.KDA_ERR_DTYPE,
                                B.KDA_ERR_UNSUPPORTED, B.KDA_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def lib():
    return P8.load_library()


def test_exports_every_declared_symbol(lib):
    src = open(os.path.join(ROOT, "include", "kda_paged_q8.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    assert set(re.findall(r"\b(kda_[a-z0-9_]+)\s*\(", src)) == set(P8.EXPORTS)
    for n in P8.EXPORTS:
        assert hasattr(lib, n), n


def test_package_exports_the_entry_points():
    import gated_delta_rule_65_amd as pkg
    assert pkg.paged_attention_q8 is P8.paged_attention_q8 and pkg.kv_append_q8 is P8.kv_append_q8
    assert pkg.kv_read_q8 is P8.kv_read_q8


def test_struct_layouts_match_the_header(tmp_path):
    structs = {"kda_kv_append_q8_args": P8.KvAppendQ8Args, "kda_kv_read_q8_args": P8.KvReadQ8Args,
               "kda_paged_attention_q8_args": P8.PagedAttentionQ8Args}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "kda_paged_q8.h"', "int main(void) {"]
    for c, py in structs.items():
        lines.append(f'printf("{c} %zu\\n", sizeof({c}));')
        lines += [f'printf("{c}.{f} %zu\\n", offsetof({c}, {f}));' for f, _ in py._fields_]
    src = tmp_path / "l.c"
    src.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "l")],
                   check=True)
    got = dict(x.split() for x in subprocess.run([str(tmp_path / "l")], capture_output=True, text=True,
                                                 check=True).stdout.splitlines())
    for c, py in structs.items():
        assert int(got[c]) == ctypes.sizeof(py)
        for f, _ in py._fields_:
            assert int(got[f"{c}.{f}"]) == getattr(py, f).offset, (c, f)


def fill(a, **kw):
    a.struct_size = ctypes.sizeof(a)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


CACHE = dict(k_cache=FAKE, v_cache=FAKE, k_scale=FAKE, v_scale=FAKE, block_table=FAKE, cu_seqlens=FAKE,
             seq_lens=FAKE, dtype=1, code=0, n=2, hkv=2, head_dim=128, page_size=16, block=8, num_pages=99,
             max_pages=8)


def append(**kw):
    return fill(P8.KvAppendQ8Args(), **{**CACHE, **dict(k=FAKE, v=FAKE, total_tokens=5), **kw})


def read(**kw):
    return fill(P8.KvReadQ8Args(), **{**CACHE, **dict(k_out=FAKE, v_out=FAKE, total_tokens=5), **kw})


def attend(**kw):
    return fill(P8.PagedAttentionQ8Args(),
                **{**CACHE, **dict(q=FAKE, out=FAKE, lse=FAKE, total_tokens=64, hq=8, scale=0.1, splits=1), **kw})


COMMON = [
    (dict(struct_size=8), ARG), (dict(dtype=7), DTYPE), (dict(code=2), DTYPE), (dict(code=-1), DTYPE),
    (dict(hkv=0), SHAPE), (dict(n=-1), SHAPE), (dict(total_tokens=-1), SHAPE), (dict(page_size=0), SHAPE),
    (dict(num_pages=0), SHAPE), (dict(max_pages=-1), SHAPE), (dict(table_stride=7), SHAPE),
    (dict(block=0), SHAPE), (dict(block=5), SHAPE), (dict(block=32), SHAPE), (dict(block=-8), SHAPE),
    (dict(head_dim=96), UNSUP), (dict(num_pages=1 << 28), UNSUP), (dict(max_pages=1 << 27), UNSUP),
    (dict(total_tokens=1 << 31), UNSUP), (dict(k_page_stride=100), SHAPE),
    (dict(v_page_stride=2 * 16 * 128 + 8), ARG), (dict(k_cache=FAKE + 8), ARG), (dict(v_cache=FAKE + 8), ARG),
    (dict(k_scale=FAKE + 2), ARG), (dict(v_scale=FAKE + 1), ARG), (dict(block_table=FAKE + 2), ARG),
    (dict(cu_seqlens=FAKE + 2), ARG), (dict(seq_lens=FAKE + 2), ARG),
    (dict(k_cache=None), ARG), (dict(v_cache=None), ARG), (dict(k_scale=None), ARG), (dict(v_scale=None), ARG),
    (dict(block_table=None), ARG), (dict(cu_seqlens=None), ARG), (dict(seq_lens=None), ARG),
]


@pytest.mark.parametrize("fields,status", COMMON + [
    (dict(k_stride=128), SHAPE), (dict(v_stride=1 << 25), SHAPE), (dict(v_stride=257), ARG),
    (dict(k=FAKE + 2), ARG), (dict(v=FAKE + 8), ARG), (dict(k=None), ARG), (dict(v=None), ARG),
    (dict(n=1 << 23), UNSUP), (dict(total_tokens=1 << 30), UNSUP), (dict(total_tokens=1 << 26), UNSUP),
])
def test_append_refusals(lib, fields, status):
    assert lib.kda_kv_append_q8(ctypes.byref(append(**fields))) == status
    assert lib.kda_last_error()


@pytest.mark.parametrize("fields,status", COMMON + [
    (dict(k_out=FAKE + 8), ARG), (dict(v_out=FAKE + 4), ARG), (dict(k_out=None), ARG), (dict(v_out=None), ARG),
    (dict(n=1 << 25), UNSUP), (dict(total_tokens=1 << 27), UNSUP),
])
def test_read_refusals(lib, fields, status):
    assert lib.kda_kv_read_q8(ctypes.byref(read(**fields))) == status
    assert lib.kda_last_error()


@pytest.mark.parametrize("fields,status", COMMON + [
    (dict(dtype=0), DTYPE), (dict(hq=0), SHAPE), (dict(hq=9), SHAPE), (dict(window=-1), SHAPE),
    (dict(sinks=-1), SHAPE), (dict(max_new_len=-1), SHAPE), (dict(splits=65), SHAPE), (dict(splits=-1), SHAPE),
    (dict(scale=float("nan")), SHAPE), (dict(scale=0.0), SHAPE), (dict(scale=2.4e38), SHAPE),
    (dict(n=1 << 24), UNSUP), (dict(q_stride=8), SHAPE), (dict(q_stride=8 * 128 + 4), ARG),
    (dict(q=FAKE + 4), ARG), (dict(out=FAKE + 8), ARG), (dict(lse=FAKE + 2), ARG), (dict(q=None), ARG),
    (dict(out=None), ARG), (dict(splits=4, max_pages=4096), WS),
    (dict(splits=4, max_pages=4096, workspace=FAKE, workspace_bytes=64), WS),
    (dict(splits=4, max_pages=4096, workspace=FAKE + 8, workspace_bytes=1 << 30), ARG),
])
def test_attention_refusals(lib, fields, status):
    assert lib.kda_paged_attention_q8(ctypes.byref(attend(**fields))) == status
    assert lib.kda_last_error()


def test_null_structs_and_empty_calls(lib):
    for fn in (lib.kda_kv_append_q8, lib.kda_kv_read_q8, lib.kda_paged_attention_q8):
        assert fn(None) == ARG
    n = ctypes.c_size_t(0)
    assert lib.kda_paged_attention_q8_workspace_size(ctypes.byref(attend()), None) == ARG
    assert lib.kda_paged_attention_q8_workspace_size(None, ctypes.byref(n)) == ARG
    for empty in (dict(total_tokens=0), dict(n=0)):
        assert lib.kda_kv_append_q8(ctypes.byref(append(k=None, v=None, **empty))) == B.KDA_OK
        assert lib.kda_kv_read_q8(ctypes.byref(read(k_out=None, **empty))) == B.KDA_OK
        assert lib.kda_paged_attention_q8(ctypes.byref(attend(q=None, out=None, **empty))) == B.KDA_OK


def test_workspace_is_bounded_and_asked_for_by_shape(lib):
    seen = []
    for dim in (64, 128):
        for hq, hkv in ((1, 1), (32, 8), (64, 1)):
            for n in (1, 4, 256):
                for hint in (0, 1):
                    for splits in (0, 2, 64):
                        for k in range(18):
                            size = ctypes.c_size_t(0)
                            a = attend(total_tokens=n + (1 << k) - 1, n=n, hq=hq, hkv=hkv, head_dim=dim,
                                       max_pages=8192, num_pages=8192, max_new_len=hint, splits=splits)
                            assert lib.kda_paged_attention_q8_workspace_size(
                                ctypes.byref(a), ctypes.byref(size)) == B.KDA_OK
                            seen.append(size.value)
    assert 0 == min(seen) < max(seen) <= P.PAGED_ATTENTION_WORKSPACE_MAX


def cpu_case(dt=torch.bfloat16, code=torch.float8_e4m3fn):
    kc = torch.zeros(5, 2, 16, 128, dtype=torch.uint8).view(code)
    ks = torch.zeros(5, 2, 2)
    cache = dict(k_cache=kc, v_cache=kc.clone(), k_scale=ks, v_scale=ks.clone(),
                 block_table=torch.zeros(2, 3, dtype=torch.int32), cu_seqlens=torch.tensor([0, 1, 3]),
                 seq_lens=torch.tensor([4, 5]))
    rows = torch.zeros(3, 2, 128, dtype=dt)
    return cache, dict(k=rows, v=rows.clone()), dict(q=torch.zeros(3, 4, 128, dtype=dt))


BAD_CACHE = [
    (dict(k_cache=torch.zeros(5, 2, 16)), ValueError, "k_cache"),
    (dict(k_cache=torch.zeros(5, 2, 16, 128)), TypeError, "k_cache"),
    (dict(k_cache=torch.zeros(5, 2, 16, 128, dtype=torch.uint8)), TypeError, "k_cache"),
    (dict(v_cache=torch.zeros(5, 2, 16, 128, dtype=torch.int8)), TypeError, "v_cache"),
    (dict(v_cache=torch.zeros(5, 2, 8, 128, dtype=torch.int8)), ValueError, "v_cache"),
    (dict(k_scale=torch.zeros(5, 2)), ValueError, "k_scale"),
    (dict(k_scale=torch.zeros(5, 2, 3)), ValueError, "k_scale"),
    (dict(k_scale=torch.zeros(5, 2, 0)), ValueError, "k_scale"),
    (dict(k_scale=torch.zeros(4, 2, 2)), ValueError, "k_scale"),
    (dict(v_scale=torch.zeros(5, 2, 4)), ValueError, "v_scale"),
    (dict(v_scale=torch.zeros(5, 2, 2, dtype=torch.float16)), TypeError, "scale"),
    (dict(v_scale=torch.zeros(5, 2, 4)[:, :, ::2]), ValueError, "contiguous"),
    (dict(block_table=torch.zeros(3, 3, dtype=torch.int32)), ValueError, "block_table"),
    (dict(block_table=torch.zeros(2, 3, dtype=torch.int64)), TypeError, "block_table"),
    (dict(cu_seqlens=torch.zeros(3, 1)), ValueError, "cu_seqlens"),
    (dict(cu_seqlens=torch.tensor([0.0, 1.0, 3.0])), TypeError, "cu_seqlens"),
    (dict(seq_lens=torch.zeros(3, dtype=torch.int32)), ValueError, "seq_lens"),
    (dict(), ValueError, "GPU"),
]


@pytest.mark.parametrize("change,exc,match", BAD_CACHE)
def test_binding_refuses_bad_caches(change, exc, match):
    cache, rows, q = cpu_case()
    with pytest.raises(exc, match=match):
        P8.kv_append_q8(**{**cache, **rows, **change})
    with pytest.raises(exc, match=match):
        P8.paged_attention_q8(**{**cache, **q, **change})
    with pytest.raises(exc, match=match):
        P8.kv_read_q8(**{**cache, **dict(total_tokens=3), **change})


def test_binding_refuses_bad_rows():
    cache, rows, q = cpu_case()
    z = torch.zeros
    for change, exc, match in (
            (dict(k=z(3, 256, dtype=torch.bfloat16)), ValueError, "k must"),
            (dict(v=z(3, 2, 64, dtype=torch.bfloat16)), ValueError, "v must"),
            (dict(k=z(3, 2, 128, dtype=torch.float64), v=z(3, 2, 128, dtype=torch.float64)), TypeError, "dtype"),
            (dict(v=z(3, 2, 128)), TypeError, "v must"),
            (dict(k=z(3, 1, 128, dtype=torch.bfloat16), v=z(3, 1, 128, dtype=torch.bfloat16)), ValueError, "k must"),
            (dict(k=z(2, 3, 128, dtype=torch.bfloat16).transpose(0, 1)), ValueError, "k must")):
        with pytest.raises(exc, match=match):
            P8.kv_append_q8(**{**cache, **rows, **change})
    for change, exc, match in (
            (dict(q=z(3, 4, 128)), TypeError, "q must"), (dict(q=z(3, 512, dtype=torch.bfloat16)), ValueError, "q must"),
            (dict(q=z(3, 5, 128, dtype=torch.bfloat16)), ValueError, "divisible"),
            (dict(q=z(3, 4, 64, dtype=torch.bfloat16)), ValueError, "k_cache"),
            (dict(window=-1), ValueError, "window"), (dict(splits=65), ValueError, "splits"),
            (dict(max_new_len=-1), ValueError, "max_new_len"),
            (dict(output=z(3, 4, 128)), TypeError, "output"), (dict(lse=z(3)), ValueError, "lse")):
        with pytest.raises(exc, match=match):
            P8.paged_attention_q8(**{**cache, **q, **change})
    for change, exc, match in (
            (dict(k_out=z(3, 2, 128)), ValueError, "together"),
            (dict(k_out=z(3, 2, 128), v_out=z(3, 2, 128, dtype=torch.bfloat16)), TypeError, "v_out"),
            (dict(k_out=z(3, 2, 64), v_out=z(3, 2, 128)), ValueError, "k_out"),
            (dict(total_tokens=-1), ValueError, "total_tokens"), (dict(dtype=torch.int8), TypeError, "dtype"),
            (dict(k_out=z(4, 2, 128), v_out=z(4, 2, 128), total_tokens=3), ValueError, "k_out")):
        with pytest.raises(exc, match=match):
            P8.kv_read_q8(**{**cache, **change})


def test_the_reference_rounds_as_torch_does():
    g = torch.Generator().manual_seed(0)
    y = torch.cat([torch.randn(4000, generator=g) * 10.0 ** torch.randint(-4, 3, (4000,), generator=g),
                   torch.from_numpy(Q.VALUES["e4m3"][:127]).float(), torch.tensor([0.0, -0.0, 2.0 ** -10, 3 * 2.0 ** -10])])
    y = y.clamp(-448, 448)
    want = y.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(Q.nearest(y.double().numpy(), "e4m3"), want)
    assert Q.least_scale(448.0, "e4m3") == 1 and Q.least_scale(448.1, "e4m3") == 2
    assert Q.least_scale(127.0, "int8") == 1 and Q.least_scale(0.0, "int8") == 2.0 ** -126


# A launch holds fewer than 2^32 threads, so fewer than 2^24 workgroups of 256.
@pytest.mark.parametrize("fields", [
    dict(n=1, hkv=1, block=16, total_tokens=((1 << 24) - 2) * 16), dict(n=2, hkv=2, block=8, total_tokens=((1 << 23) - 4) * 8),
    dict(n=1 << 22, hkv=2, block=16, total_tokens=1), dict(n=3, hkv=5, block=16, total_tokens=((1 << 24) // 5 + 1 - 6) * 16)])
def test_appends_past_a_launch_are_unsupported(lib, fields):
    assert lib.kda_kv_append_q8(ctypes.byref(append(**fields))) == UNSUP
    assert b"2^24" in lib.kda_last_error()


@pytest.mark.parametrize("fields", [dict(n=2, total_tokens=((1 << 24) - 2) * 4), dict(n=(1 << 24) - 1, total_tokens=4), dict(n=1 << 24, total_tokens=1)])
def test_reads_past_a_launch_are_unsupported(lib, fields):
    assert lib.kda_kv_read_q8(ctypes.byref(read(**fields))) == UNSUP
    assert b"2^26" in lib.kda_last_error()
