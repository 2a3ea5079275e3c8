"""The rotary positions on the host: exports, struct agreement, argument checks of the C ABI and of
the binding, and the frequencies against their formulas.  No call here gets as far as queueing work."""
import ctypes
import math
import os
import re
import subprocess

import pytest
import torch

from gated_delta_rule_65_amd import binding as B
from gated_delta_rule_65_amd import positions as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20      # a well-aligned address that no check reads through
ARG, SHAPE, DTYPE, UNSUP = B.KDA_ERR_ARG, B.KDA_ERR_SHAPE, B.KDA_ERR_DTYPE, B.KDA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    return R.load_library()


def test_exports_every_declared_symbol(lib):
    src = open(os.path.join(ROOT, "include", "kda_rotary.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    assert set(re.findall(r"\b(kda_[a-z0-9_]+)\s*\(", src)) == set(R.EXPORTS)
    import gated_delta_rule_65_amd as pkg
    assert pkg.rotary is R.rotary and pkg.rotary_frequencies is R.rotary_frequencies


def test_struct_layout_matches_the_header(tmp_path):
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "kda_rotary.h"', "int main(void) {",
             'printf("size %zu\\n", sizeof(kda_rotary_args));']
    lines += [f'printf("{f} %zu\\n", offsetof(kda_rotary_args, {f}));' for f, _ in R.RotaryArgs._fields_]
    src = tmp_path / "l.c"
    src.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "l")],
                   check=True)
    got = dict(x.split() for x in subprocess.run([str(tmp_path / "l")], capture_output=True, text=True,
                                                 check=True).stdout.splitlines())
    assert int(got["size"]) == ctypes.sizeof(R.RotaryArgs)
    for f, _ in R.RotaryArgs._fields_:
        assert int(got[f]) == getattr(R.RotaryArgs, f).offset, f


MB = 1 << 20


def args(**kw):
    d = dict(q=MB, k=2 * MB, q_out=3 * MB, k_out=4 * MB, positions=5 * MB, frequencies=6 * MB, total_tokens=5,
             dtype=1, hq=4, hk=2, head_dim=128, pairs=64, scale=1.0)
    d.update(kw)
    a = R.RotaryArgs()
    a.struct_size = ctypes.sizeof(a)
    for k, v in d.items():
        setattr(a, k, v)
    return a


ROW = 4 * 128 * 2      # bytes of a token of q


@pytest.mark.parametrize("fields,status", [
    (dict(struct_size=8), ARG), (dict(dtype=5), DTYPE), (dict(dtype=-1), DTYPE), (dict(total_tokens=-1), SHAPE),
    (dict(hq=0), SHAPE), (dict(hk=0), SHAPE), (dict(head_dim=0), SHAPE), (dict(head_dim=12), UNSUP),
    (dict(head_dim=520), UNSUP), (dict(pairs=0), SHAPE), (dict(pairs=65), SHAPE),
    (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE), (dict(q_stride=8), SHAPE),
    (dict(k_stride=1 << 25), SHAPE), (dict(q_out_stride=4 * 128 + 4), ARG), (dict(k_out_stride=8), SHAPE),
    (dict(total_tokens=1 << 40), UNSUP), (dict(q=MB + 2), ARG), (dict(k_out=4 * MB + 8), ARG),
    (dict(positions=5 * MB + 2), ARG), (dict(frequencies=6 * MB + 4), ARG), (dict(q=None), ARG),
    (dict(q_out=None), ARG), (dict(k_out=None), ARG), (dict(positions=None), ARG), (dict(frequencies=None), ARG),
    # shared memory: shifted by a row, at another stride, with the other tensor, with the lists
    (dict(q_out=MB + ROW), ARG), (dict(q_out=MB - ROW), ARG), (dict(q_out=MB + 16), ARG),
    (dict(q_out=MB, q_out_stride=1024), ARG), (dict(q_out=2 * MB), ARG), (dict(k_out=MB), ARG),
    (dict(k_out=3 * MB), ARG), (dict(k_out=3 * MB + 16), ARG), (dict(q_out=5 * MB), ARG),
    (dict(k_out=6 * MB), ARG), (dict(positions=3 * MB + 5 * ROW - 4), ARG),
    # columns of one wider array that overlap
    (dict(q_stride=2048, q_out=MB + ROW - 16, q_out_stride=2048), ARG),
    (dict(q_stride=2048, q_out=MB + 2 * 4096 - ROW + 16, q_out_stride=2048), ARG),
])
def test_refusals(lib, fields, status):
    assert lib.kda_rotary(ctypes.byref(args(**fields))) == status
    assert lib.kda_last_error()


def test_null_struct_and_empty_call(lib):
    assert lib.kda_rotary(None) == ARG
    assert lib.kda_rotary(ctypes.byref(args(total_tokens=0, q=None, k=None, positions=None))) == B.KDA_OK


def test_binding_refusals():
    z = torch.zeros
    q, k = z(3, 4, 128, dtype=torch.bfloat16), z(3, 2, 128, dtype=torch.bfloat16)
    pos, f = z(3, dtype=torch.int32), z(32, dtype=torch.float64)
    for a, kw, exc, match in (
            ((q[0], k, pos, f), {}, ValueError, "q must"), ((q.double(), k, pos, f), {}, TypeError, "dtype"),
            ((q, k[:2], pos, f), {}, ValueError, "k must"), ((q, k[..., :64], pos, f), {}, ValueError, "k must"),
            ((q, k.float(), pos, f), {}, TypeError, "k must"), ((q, k, pos[:2], f), {}, ValueError, "positions"),
            ((q, k, pos.long(), f), {}, TypeError, "positions"), ((q, k, pos, f.float()), {}, TypeError, "frequencies"),
            ((q, k, pos, z(65, dtype=torch.float64)), {}, ValueError, "frequencies"),
            ((q, k, pos, z(0, dtype=torch.float64)), {}, ValueError, "frequencies"),
            ((q, k, pos, z(64, dtype=torch.float64)[::2]), {}, ValueError, "contiguous"),
            ((q, None, pos, f), dict(k_out=k), ValueError, "k_out"),
            ((q, k, pos, f), dict(q_out=q[:2]), ValueError, "q_out"),
            ((q, k, pos, f), dict(k_out=k.float()), TypeError, "k_out"),
            ((q.transpose(0, 1).contiguous().transpose(0, 1), k, pos, f), {}, ValueError, "q must"),
            ((q, k, pos, f), {}, ValueError, "GPU")):
        with pytest.raises(exc, match=match):
            R.rotary(*a, **kw)


def test_frequencies_follow_their_formulas():
    f = R.rotary_frequencies(64)
    assert f.dtype is torch.float64 and f.shape == (32,)
    for i in (0, 1, 17, 31):
        assert f[i] == pytest.approx(10000.0 ** (-2 * i / 64), rel=1e-14)
    assert torch.equal(R.rotary_frequencies(64, scaling="linear", factor=8.0), f / 8)
    b = R.rotary_frequencies(64, scaling="base", factor=8.0)
    assert b[0] == 1 and b[-1] == pytest.approx(float(f[-1]) / 8, rel=1e-12)
    t = R.rotary_frequencies(128, base=500000.0, scaling="turns", factor=16.0, original_length=8192)
    plain = R.rotary_frequencies(128, base=500000.0)
    turns = 8192 * plain / (2 * math.pi)
    # the ramp's ends are rounded outward to whole pairs
    assert torch.equal(t[turns >= 33], plain[turns >= 33])
    assert torch.allclose(t[turns <= 0.8], plain[turns <= 0.8] / 16, rtol=1e-14)
    ratio = plain / t
    assert torch.all(ratio[1:] >= ratio[:-1] - 1e-12)
    mid = ratio[(turns > 2) & (turns < 16)]     # inside the ramp from 32 turns to 1
    assert mid.numel() > 5 and torch.all((mid > 1) & (mid < 16))
    # a factor of 1 changes nothing
    for s in ("linear", "base", "turns"):
        assert torch.allclose(R.rotary_frequencies(64, scaling=s, original_length=4096), f, rtol=1e-14)


def test_pairs_of_many_turns_are_not_divided_in_full():
    # 32 channels over 10^6 positions: every pair makes more than a turn (the slowest 28), so
    # none is divided by the whole factor, and the ramp runs from 32 turns (pair 14.8) to 1 (pair 20.8)
    plain = R.rotary_frequencies(32)
    t = R.rotary_frequencies(32, scaling="turns", factor=8.0, original_length=10 ** 6)
    assert torch.equal(t[:15], plain[:15])
    slow = (15 - 14) / (21 - 14)        # of the last pair, the ends rounded outward
    assert float(t[15]) == pytest.approx(float(plain[15]) * (1 - slow + slow / 8), rel=1e-12)
    # over 10 positions no pair makes 32 turns: the ramp starts at the first pair
    t = R.rotary_frequencies(32, scaling="turns", factor=8.0, original_length=10)
    # and ends at pair 0.8, rounded up
    assert t[0] == plain[0]
    assert torch.allclose(t[1:], plain[1:] / 8, rtol=1e-14)


@pytest.mark.parametrize("a,kw", [
    ((63,), {}), ((0,), {}), ((64,), dict(base=-1.0)), ((64,), dict(base=float("inf"))),
    ((64,), dict(factor=0.0)), ((64,), dict(scaling="other")), ((2,), dict(scaling="base", factor=2.0)),
    ((64,), dict(scaling="turns", factor=2.0)), ((64,), dict(scaling="turns", original_length=0)),
    ((64,), dict(scaling="turns", original_length=100, slow_turns=3, fast_turns=2)),
    ((64,), dict(scaling="turns", original_length=100, base=1.0)),
    ((64,), dict(scaling="turns", original_length=100, base=0.5)),
])
def test_frequencies_refuse(a, kw):
    with pytest.raises(ValueError):
        R.rotary_frequencies(*a, **kw)


@pytest.mark.parametrize("fields", [
    # a launch holds fewer than 2^32 threads: workgroups of 256, four tokens each
    dict(total_tokens=1 << 26), dict(total_tokens=(1 << 26) - 3), dict(total_tokens=1 << 28), dict(total_tokens=(1 << 26) + 1, dtype=0)])
def test_tokens_past_a_launch_are_unsupported(lib, fields):
    a = args(**{**dict(hq=1, hk=0, k=None, k_out=None, head_dim=8, pairs=4, q=1 << 40, q_out=1 << 50), **fields})
    assert lib.kda_rotary(ctypes.byref(a)) == UNSUP
    assert b"2^26" in lib.kda_last_error()
