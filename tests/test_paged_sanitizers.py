"""The paged operators' host-side argument checks under AddressSanitizer and
UndefinedBehaviorSanitizer, on the CPU: kda_paged_api.hip is rebuilt with host-only
sanitizer flags, linked with the regular build's other objects, and
tests/test_paged_cpu.py runs against that library with the sanitizer runtime
preloaded.  Device code is built as usual; no GPU call is made.
"""
import glob
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gated_delta_rule_65_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ASAN_RT = sorted(glob.glob("/opt/rocm/llvm/lib/clang/*/lib/linux/libclang_rt.asan-x86_64.so"))


def _run(cmd, **kw):
    r = subprocess.run(cmd, capture_output=True, text=True, **kw)
    assert r.returncode == 0, f"{cmd[0]} exited {r.returncode}:\n{r.stdout[-4000:]}\n{r.stderr[-4000:]}"
    return r


def test_paged_host_checks_under_asan_ubsan(tmp_path):
    sources = sorted(os.path.basename(s) for s in glob.glob(os.path.join(CSRC, "*.hip")))
    objs = [os.path.join(ROOT, "_build", s + ".o") for s in sources if s != "kda_paged_api.hip"]
    missing = [o for o in objs if not os.path.exists(o)]
    if missing or not ASAN_RT or not os.path.exists(HIPCC):
        pytest.skip(f"needs the regular build's objects ({missing}), hipcc and clang's ASan runtime")
    api_o, lib = str(tmp_path / "api.o"), str(tmp_path / "libkda_asan.so")
    host = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
            "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer"]
    _run([HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-fvisibility=hidden",
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-I", os.path.join(ROOT, "include"), "-I", CSRC, *host,
          "-c", os.path.join(CSRC, "kda_paged_api.hip"), "-o", api_o])
    _run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", api_o, *objs,
          "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
          "-shared-libsan", "-o", lib])
    env = dict(os.environ, LD_PRELOAD=ASAN_RT[-1], KDA_LIBRARY=lib,
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1")
    r = _run(["python", "-m", "pytest", os.path.join(ROOT, "tests", "test_paged_cpu.py"), "-x", "-q",
              "-p", "no:cacheprovider"], env=env, cwd=ROOT, timeout=900)
    assert " passed" in r.stdout
