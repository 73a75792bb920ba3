"""Which kernel and how many K splits the routed-expert planner gives (CPU; tests/experts_plan_query.cpp
built with awq_plan.cpp)."""
from __future__ import annotations

import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GATE_UP, DOWN, MLP = 1, 2, 3
CUS = 256


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    """plans([(T, topk, E, K, inner, N, group_size, halves), ...]) -> a dict of each product per call."""
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("plan") / "query")
    cmd = [cxx, "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", os.path.join(ROOT, "tests", "experts_plan_query.cpp"),
           os.path.join(ROOT, "w4a16_weight_only_amd", "csrc", "awq_plan.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    keys = ("stream", "ranked", "rows", "tiles", "col_tiles", "splits", "grid")

    def ask(cases):
        text = "\n".join(" ".join(map(str, (*c[:7], CUS, c[7]))) for c in cases)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=300).stdout.splitlines()
        assert len(out) == len(cases)
        v = [list(map(int, line.split())) for line in out]
        assert all(x[0] == 0 for x in v), [c for c, x in zip(cases, v) if x[0] != 0][:3]
        return [dict(two_terms=x[1], up=dict(zip(keys, x[2:9])), down=dict(zip(keys, x[9:16]))) for x in v]

    return ask


def test_entries_of_one_expert_count_as_workgroups(plans):
    """An expert's rows are several entries of 32, each with workgroups of its own: where those fill
    the card, K is not split."""
    got = plans([(T, 1, 1, 4096, 4096, 4096, 128, DOWN) for T in (64, 256, 512, 1024)])
    assert [p["down"]["splits"] for p in got] == [8, 2, 1, 1]


def test_no_splits_where_entries_fill_the_card(plans):
    """Streamed products whose full entries alone are eight workgroups per compute unit and more."""
    rng = random.Random(3)
    cases = []
    while len(cases) < 4000:
        E, topk = rng.choice(((1, 1), (8, 2), (20, 4), (64, 8), (128, 8)))
        K, N = 128 * rng.randint(4, 120), 128 * rng.randint(4, 120)
        cases.append((rng.randint(1, 4000), topk, E, 0, K, N, 128, DOWN))
    filled = 0
    for c, p in zip(cases, plans(cases)):
        d = p["down"]
        if d["stream"] and c[0] * c[1] // d["rows"] * d["col_tiles"] >= 8 * CUS:
            filled += 1
            assert d["splits"] == 1, (c, d)
    assert filled > 100


def test_family_by_row_tiles(plans):
    """Row tiles from a third of the card's workgroups on: the second product of prompts through
    8 x 4096 -> 14336, one dense expert."""
    got = plans([(T, 2, 8, 4096, 14336, 4096, 128, MLP) for T in (200, 320, 512, 768, 1024)])
    assert [(p["up"]["stream"], p["down"]["stream"]) for p in got] == [(1, 1), (0, 1), (0, 1), (0, 0), (0, 0)]
    got = plans([(T, 1, 1, 0, 4096, 4096, 128, DOWN) for T in (64, 1024, 2048)])
    assert [p["down"]["stream"] for p in got] == [1, 1, 0]


def test_families_of_the_gpu_tests(plans):
    """The GPU tests of row tiles, and of both kernels in one call, run what they say."""
    from tests import expert_sizes as sizes

    for counts in sizes.HEIGHTS:
        S, E = sum(counts), len(counts)
        for K, g in sizes.HEIGHT_KS:
            p, q = plans([(S, 1, E, K, sizes.HEIGHT_INNER, 0, g, GATE_UP), (S, 1, E, 0, K, sizes.HEIGHT_N, g, DOWN)])
            assert not p["up"]["stream"] and not q["down"]["stream"], (counts, K)
    for (T, E, topk, K, inner, N, g), up, down in sizes.FAMILIES:
        p = plans([(T, topk, E, K, inner, N, g, MLP)])[0]
        assert (p["up"]["stream"], p["down"]["stream"]) == (up, down) and not p["two_terms"], (T, E, inner, N)
