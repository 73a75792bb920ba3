"""Host-only sanitizer build of the routed-expert planner (CPU): awq_plan.cpp with
tests/experts_plan_check.cpp under AddressSanitizer and UndefinedBehaviorSanitizer, a sweep
of sizes from the limits and beyond to random layers, each plan checked against the
kernels' contracts."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_experts_planner_sweep_under_asan_ubsan(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "experts_plan_check")
    cmd = [cxx, "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-static-libasan", "-static-libubsan", "-Wall", "-Wextra", "-Werror",
           os.path.join(ROOT, "tests", "experts_plan_check.cpp"),
           os.path.join(ROOT, "w4a16_weight_only_amd", "csrc", "awq_plan.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    print(r.stdout, r.stderr[-4000:])
    assert r.returncode == 0, r.stderr[-4000:]
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr
    assert int(r.stdout.split("plans checked:")[1].split()[0]) > 1_000_000
