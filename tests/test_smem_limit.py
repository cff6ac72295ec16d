"""The shared-memory limit of kernels whose size changes from call to call,
asked for by two host threads at once: compiles tests/native/smem_check.cpp as
host code and runs it on the CPU (see the file)."""
import pathlib
import subprocess

import pytest

from w4_weight_only_b200 import build

ROOT = pathlib.Path(__file__).resolve().parents[1]


def test_two_threads_and_two_sizes(tmp_path):
    try:
        nvcc = build.nvcc_path()
    except RuntimeError:
        pytest.skip("nvcc not found")
    exe = tmp_path / "smem_check"
    # (without the runtime library: the file has its own form of the calls)
    cmd = [nvcc, "-std=c++17", "-O1", "-cudart", "none", "-I", str(ROOT / "include"),
           "-I", str(ROOT / "w4_weight_only_b200" / "csrc"), str(ROOT / "tests" / "native" / "smem_check.cpp"),
           "-Xcompiler", "-pthread", "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0 and "smem ok" in out.stdout, out.stdout[-2000:]
