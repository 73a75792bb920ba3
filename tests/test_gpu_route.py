"""awq_moe_route against the oracle in float64.

ids must be equal.  Weights: fp32, formed as exp(a) / sum of exp(b) (softmax), or with one
more quotient each (sigmoid), times scale.  Relative error, in units of 2^-24 (half a step of
fp32): the argument of exp is a difference rounded once, at most 40 here for weights that
matter, so exp is off by 40 from it and 2 of its own; a sum of n positive terms adds at most
one per term on the longest path (n / 64 + 7 for n experts over 64 lanes); divisions and
products add 4.  Together under 40 + 2 + (40 + 2 + 23) + 8 = 115, that is 7e-6; an absolute
1e-30 covers scores too small for fp32.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import w4a16_weight_only_amd as awq
from oracle import awq_ref as oracle

pytestmark = pytest.mark.gpu

RTOL, ATOL = 7e-6, 1e-30


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a HIP GPU")
    awq.load_library()


def check(logits, topk, bias=None, out=None, **kw):
    """Runs the operator on device logits and compares with the oracle on the same values."""
    print(f"route {tuple(logits.shape)} {logits.dtype} topk={topk} bias={bias is not None} {kw}", flush=True)
    w, i = awq.awq_moe_route(logits, topk, bias=bias, out=out, **kw)
    torch.cuda.synchronize()
    wr, ir = oracle.route_ref(logits.double().cpu().numpy(), topk,
                              bias=None if bias is None else bias.double().cpu().numpy(), **kw)
    assert w.dtype == torch.float32 and i.dtype == torch.int32
    assert np.array_equal(i.cpu().numpy(), ir)
    np.testing.assert_allclose(w.cpu().numpy(), wr, rtol=RTOL, atol=ATOL)
    return w, i


def normal(T, E, dtype, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) * spread).to(dtype).cuda()


def normal_bias(E, seed=1):
    return (0.2 * torch.randn(E, generator=torch.Generator().manual_seed(seed))).cuda()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,topk", [(1, 1, 1), (1, 8, 2), (3, 60, 4), (2, 64, 64), (65, 65, 8), (33, 128, 8),
                                       (7, 200, 1), (5, 256, 8), (9, 257, 10), (4, 512, 16), (3, 1000, 33),
                                       (2, 1024, 64)])
def test_plain(T, E, topk, score, dtype):
    logits = normal(T, E, dtype, T * E + topk)
    check(logits, topk, score=score)
    check(logits, topk, score=score, renormalize=False, scale=2.5)
    check(logits, topk, bias=normal_bias(E), score=score, scale=0.5)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,groups,topk_groups,topk", [(5, 8, 8, 3, 3), (65, 60, 5, 2, 7), (9, 256, 8, 4, 8),
                                                        (3, 64, 64, 9, 9), (4, 96, 3, 3, 11), (2, 1024, 16, 1, 64),
                                                        (6, 512, 64, 32, 8), (1, 14, 2, 1, 7)])
def test_groups(T, E, groups, topk_groups, topk, score, dtype):
    logits = normal(T, E, dtype, T + E)
    for group_top in (1, 2):
        for bias in (None, normal_bias(E)):
            check(logits, topk, bias=bias, score=score, groups=groups, topk_groups=topk_groups, group_top=group_top)


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_go_to_the_lowest_index(score, group_top, biased):
    """Few distinct logits, so that experts and whole groups tie, with and without an equal bias."""
    g = torch.Generator().manual_seed(5)
    logits = torch.randint(-1, 2, (50, 48), generator=g).to(torch.float16).cuda()
    bias = torch.full((48,), 0.25).cuda() if biased else None
    check(logits, 6, bias=bias, score=score)
    check(logits, 6, bias=bias, score=score, groups=6, topk_groups=2, group_top=group_top)
    check(torch.zeros(3, 48, device="cuda"), 5, bias=bias, score=score, groups=4, topk_groups=1, group_top=group_top)


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_experts(score, biased):
    """-inf logits are never chosen: rows with fewer left than topk, with one, with none, and
    groups of which nothing or one is left; the types' lowest values still are choices."""
    E = 40
    logits = normal(8, E, torch.float32, 11)
    logits[0] = -float("inf")
    logits[1, 1:] = -float("inf")
    logits[2, 3:] = -float("inf")
    logits[3, ::2] = -float("inf")
    logits[4, :30] = -float("inf")
    logits[5] = torch.finfo(torch.float32).min
    logits[6, 1:] = torch.finfo(torch.float32).min
    logits[7, :20] = -float("inf")
    logits[7, 21:30] = -float("inf")
    bias = normal_bias(E) if biased else None
    for kw in ({}, dict(renormalize=False), dict(groups=4, topk_groups=2), dict(groups=4, topk_groups=2, group_top=2),
               dict(groups=4, topk_groups=4, group_top=2)):
        check(logits, 6, bias=bias, score=score, **kw)
    half = logits.clamp(min=torch.finfo(torch.float16).min).half()
    check(half, 6, bias=bias, score=score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_nonfinite_rows(score):
    """NaN anywhere, +inf, and their neighbours, which must not notice."""
    logits = normal(6, 24, torch.float32, 12)
    logits[1, 23] = float("nan")
    logits[2, 5] = float("inf")
    logits[4] = float("nan")
    check(logits, 3, score=score)
    check(logits, 3, score=score, groups=3, topk_groups=2)
    check(logits, 3, score=score, bias=normal_bias(24))


def test_bias_that_masks_or_forces():
    bias = normal_bias(16)
    bias[3] = -float("inf")
    bias[7] = float("inf")
    logits = normal(9, 16, torch.float16, 13)
    logits[0, 7] = -float("inf")  # a masked expert stays masked, whatever its bias
    check(logits, 15, score="sigmoid", bias=bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("shift", [-300.0, -90.0, 0.0, 90.0, 300.0])
def test_far_logits(score, shift):
    """Scores that fp32 cannot hold still divide (and saturated ones still have an order)."""
    logits = normal(5, 32, torch.float32, 14) + shift
    check(logits, 4, score=score)
    check(logits, 4, score="softmax", renormalize=False)


def test_close_scores_keep_their_order():
    """Sigmoid + bias sums that differ by less than fp32 resolves: the order is the fp64 one."""
    E = 64
    base = torch.full((1, E), 1.0, dtype=torch.float32)
    logits = base.cuda().repeat(4, 1)
    bias = torch.zeros(E)
    logits[:, 1::2] += 2.0 ** -22  # score larger by 0.2 * 2^-22 in the odd experts
    bias[::2] = 2.0 ** -25         # less than that in the even ones
    w, i = check(logits, 8, score="sigmoid", bias=bias.cuda())
    assert (i.cpu()[0] % 2 == 1).all()


def test_strided_rows_and_out():
    """A column range of a wider matrix; outputs written in place, nothing around them."""
    wide = normal(21, 100, torch.bfloat16, 15)
    view = wide[:, 7:71]
    w = torch.full((22, 4), 5.0, device="cuda")
    i = torch.full((22, 4), 9, dtype=torch.int32, device="cuda")
    check(view, 4, out=(w[:21], i[:21]))
    assert (w[21] == 5).all() and (i[21] == 9).all()
    assert awq.awq_moe_route(wide[:0], 4)[1].shape == (0, 4)


def test_many_tokens():
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.randn(5000, 72, device="cuda", generator=g)
    check(logits, 6, score="sigmoid", bias=normal_bias(72), groups=8, topk_groups=3, group_top=2)


def test_streams_and_graphs():
    logits = normal(300, 128, torch.float16, 16)
    bias = normal_bias(128)
    ref = awq.awq_moe_route(logits, 8, score="sigmoid", bias=bias)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        got = awq.awq_moe_route(logits, 8, score="sigmoid", bias=bias)
    other.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    out = tuple(torch.zeros_like(t) for t in ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        awq.awq_moe_route(logits, 8, score="sigmoid", bias=bias, out=out)
    for _ in range(3):
        logits.add_(0.5)
        want = awq.awq_moe_route(logits, 8, score="sigmoid", bias=bias)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_refusals():
    logits = normal(4, 16, torch.float16, 17)
    for bad in (dict(topk=0), dict(topk=17), dict(topk=4, groups=3), dict(topk=9, groups=2, topk_groups=1),
                dict(topk=2, group_top=0), dict(topk=2, score="relu"), dict(topk=2, bias=torch.zeros(15, device="cuda")),
                dict(topk=2, out=(torch.zeros(4, 3, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda")))):
        with pytest.raises(ValueError):
            awq.awq_moe_route(logits, **bad)
    with pytest.raises(ValueError):
        awq.awq_moe_route(logits.t(), 2)
    with pytest.raises(ValueError):
        awq.awq_moe_route(logits[0], 2)
    with pytest.raises(TypeError):
        awq.awq_moe_route(logits, 2, bias=torch.zeros(16, device="cuda", dtype=torch.float16))
