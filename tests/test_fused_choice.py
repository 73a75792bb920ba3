"""awq_gemm_fused's choice between streaming with K splits and row tiles, on the CPU, against measured times (fp16, us)
at sizes where splits of 32-row blocks would take several rounds of workgroups."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# (M, K, N, g, gated): {(tile height, or 0 streamed, K splits): us}
MEASURED = {
    (300, 2048, 8192, 64, 0): {(0, 1): 38.2, (0, 2): 46, (0, 4): 64.8, (192, 4): 36.4, (192, 3): 36.5, (256, 4): 37.6},
    (384, 2048, 8192, 64, 0): {(0, 1): 37.9, (0, 2): 47.5, (192, 3): 38.3, (128, 2): 38.9},
    (73, 4096, 11008, 128, 1): {(0, 3): 53.1, (0, 4): 52.5, (0, 1): 54, (128, 2): 47.7, (128, 5): 52.4},
    (96, 4096, 11008, 128, 1): {(0, 3): 59.8, (0, 1): 55.0, (128, 2): 48.6, (128, 4): 56.4},
    (73, 8192, 8192, 128, 0): {(0, 8): 48.9, (0, 2): 34.0, (128, 8): 34.3, (128, 7): 36.9},
    (96, 8192, 8192, 128, 0): {(0, 8): 55.2, (0, 2): 34.8, (128, 8): 35.2, (128, 7): 37.8},
    (160, 8192, 8192, 128, 0): {(0, 3): 57.0, (256, 8): 47.0, (192, 8): 47.2, (192, 7): 48.1},
    (73, 5120, 13824, 128, 1): {(0, 3): 64.1, (128, 2): 58.9, (128, 4): 64.8},
    (96, 5120, 13824, 128, 1): {(0, 3): 71.9, (0, 1): 70.3, (128, 2): 59.1, (128, 4): 68.1},
}


def test_splits_over_several_rounds(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "around_plan_check")
    r = subprocess.run([cxx, "-std=c++17", "-O1", os.path.join(ROOT, "tests", "around_plan_check.cpp"),
                        os.path.join(ROOT, "w4a16_weight_only_amd", "csrc", "awq_plan.cpp"), "-o", exe],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    asked = "\n".join(" ".join(map(str, case)) for case in MEASURED)
    out = subprocess.run([exe, "query"], input=asked, capture_output=True, text=True, timeout=60).stdout.splitlines()
    for (case, times), line in zip(MEASURED.items(), out):
        status, stream, rows, splits = map(int, line.split())
        chosen = (0 if stream else rows, splits)
        assert status == 0 and times.get(chosen, 1e9) <= 1.1 * min(times.values()), (case, chosen)
