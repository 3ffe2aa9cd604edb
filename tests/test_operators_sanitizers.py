"""The C entry points of the norm, the grouped products and clipping, and the
products' host rules, under AddressSanitizer and UndefinedBehaviorSanitizer
(no GPU, no device code): tests/c/sanitize_ops.cpp drives api_ops.cpp with
ordinary, degenerate and extreme arguments, the kernel launchers replaced by
host stand-ins."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SAN = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer",
       "-g", "-O1"]


def _run(cmd, **kw):
    r = subprocess.run(cmd, capture_output=True, text=True, **kw)
    assert r.returncode == 0, f"{' '.join(cmd)}\n{r.stdout}\n{r.stderr}"
    return r


@pytest.mark.skipif(shutil.which("g++") is None, reason="host compiler not found")
def test_operator_entry_points_under_asan_ubsan(tmp_path):
    inc = ["-I", os.path.join(ROOT, "include"), "-I", "/opt/rocm/include",
           "-D__HIP_PLATFORM_AMD__"]
    objs = []
    for src in ("block_sparse_gemm_amd/csrc/api.cpp", "block_sparse_gemm_amd/csrc/api_ops.cpp",
                "block_sparse_gemm_amd/csrc/grouped_plan.cpp", "tests/c/sanitize_stubs.cpp",
                "tests/c/sanitize_ops.cpp"):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        _run(["g++", "-std=c++17", *SAN, *inc, "-c", os.path.join(ROOT, src), "-o", obj])
        objs.append(obj)
    exe = str(tmp_path / "sanitize_ops")
    _run(["g++", *SAN, *objs, "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out
    assert "runtime error" not in out and "AddressSanitizer" not in out, out
    assert "sanitized operator checks passed" in out
