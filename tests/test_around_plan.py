"""The planners of awq_gemm_fused and awq_moe_layer on the CPU: a sweep under AddressSanitizer and
UndefinedBehaviorSanitizer, and which kernel the GPU tests' sizes reach."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

from tests.fused_sizes import GATED_TILES, TILES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("plan") / "around_plan_check")
    cmd = [cxx, "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-static-libasan", "-static-libubsan", "-Wall", "-Wextra", "-Werror",
           os.path.join(ROOT, "tests", "around_plan_check.cpp"),
           os.path.join(ROOT, "w4a16_weight_only_amd", "csrc", "awq_plan.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    return exe


def test_sweep(program):
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([program], capture_output=True, text=True, timeout=300, env=env)
    print(r.stdout, r.stderr[-4000:])
    assert r.returncode == 0, r.stderr[-4000:]
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr
    assert int(r.stdout.split("plans checked:")[1].split()[0]) >= 800_000


def ask(program, cases):
    text = "\n".join(" ".join(map(str, c)) for c in cases)
    out = subprocess.run([program, "query"], input=text, capture_output=True, text=True, timeout=60).stdout.splitlines()
    return [tuple(map(int, line.split())) for line in out]


@pytest.mark.parametrize("gated,sizes", [(0, TILES), (1, GATED_TILES)], ids=["plain", "gated"])
def test_sizes_reach_their_kernels(program, gated, sizes):
    for (height, split), cases in sizes.items():
        for case, (status, stream, rows, splits) in zip(cases, ask(program, [c + (gated,) for c in cases])):
            assert (status, stream, rows, splits > 1) == (0, 0, height, split), case


def test_measured_choices(program):
    """Few rows stream, many take row tiles, at the sizes that decided it."""
    cases = [(1, 4096, 4096, 128, 0), (500, 4096, 4096, 128, 0), (200, 2048, 8192, 64, 0), (750, 4096, 4096, 128, 0),
             (200, 11008, 4096, 128, 0), (1000, 11008, 4096, -1, 0), (500, 4096, 11008, 128, 1), (2048, 4096, 11008, 128, 1)]
    got = ask(program, cases)
    assert [bool(stream) for _, stream, _, _ in got] == [True, True, True, False, False, False, False, False], got
