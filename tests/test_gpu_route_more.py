"""awq_moe_route where scores of different logits round to the same number.

Same comparison and tolerances as test_gpu_route.py; of thousands of tokens the oracle, which takes
one at a time, does the last sixteen, fifty others and those that a test names."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import w4a16_weight_only_amd as awq
from oracle import awq_ref as oracle
from tests.test_gpu_route import ATOL, RTOL, check, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a HIP GPU")
    awq.load_library()


def check_some(logits, topk, also=(), bias=None, **kw):
    T = logits.shape[0]
    if T <= 2048:
        return check(logits, topk, bias=bias, **kw)
    print(f"route {tuple(logits.shape)} {logits.dtype} topk={topk} bias={bias is not None} {kw}", flush=True)
    w, i = awq.awq_moe_route(logits, topk, bias=bias, **kw)
    torch.cuda.synchronize()
    rows = np.unique([*also, *range(T - 16, T), *np.random.default_rng(T + topk).integers(0, T, 50)])
    wr, ir = oracle.route_ref(logits.double().cpu().numpy()[rows], topk,
                              bias=None if bias is None else bias.double().cpu().numpy(), **kw)
    assert np.array_equal(i.cpu().numpy()[rows], ir)
    np.testing.assert_allclose(w.cpu().numpy()[rows], wr, rtol=RTOL, atol=ATOL)
    return w, i


@pytest.mark.parametrize("T", [5, 2051])
@pytest.mark.parametrize("score,shift", [("sigmoid", 60.0), ("sigmoid", -900.0), ("softmax", 0.0)])
@pytest.mark.parametrize("E,groups,topk_groups,topk", [(8, 2, 2, 3), (48, 6, 6, 7), (256, 8, 8, 8), (60, 5, 5, 9),
                                                      (1024, 16, 16, 20)])
def test_groups_of_two_choose_by_the_logits(E, groups, topk_groups, topk, score, shift, T):
    """All groups stay, so the choice is that of the largest logits, whose scores round to 1.0, to the
    same subnormal or (softmax, one logit far above the others) to 0.0."""
    logits = normal(T, E, torch.float32, E + T, spread=5.0) + shift
    if score == "softmax":
        logits[:, E // 2] += 1500.0
    _, ids = check_some(logits, topk, score=score, groups=groups, topk_groups=topk_groups, group_top=2)
    want = np.argsort(-logits.cpu().numpy(), axis=1, kind="stable")[:, :topk]
    assert np.array_equal(ids.cpu().numpy(), want)


# More than 2048 tokens, where four of them share a wave (up to 128 experts, or 256 compared by
# their logits); not a multiple of four, so that the last wave has lanes without a token.
DTYPES = pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])


def bias_of(E, seed=1):
    return (0.2 * torch.randn(E, generator=torch.Generator().manual_seed(seed))).cuda()


@DTYPES
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,topk", [(1, 1), (8, 2), (9, 9), (64, 8), (72, 33), (100, 64), (128, 8), (200, 20), (256, 8),
                                    (256, 64), (257, 3)])
def test_many_tokens_without_groups(E, topk, score, dtype):
    T = 2050 + E % 3
    logits = normal(T, E, dtype, T + topk)
    check_some(logits, topk, score=score)
    check_some(logits, topk, score=score, renormalize=False, scale=2.5)
    check_some(logits, topk, score=score, bias=bias_of(E))


@DTYPES
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,topk_groups,topk", [(8, 2, 1, 3), (64, 8, 4, 8), (64, 64, 17, 17), (72, 9, 3, 11),
                                                      (128, 32, 20, 33), (256, 8, 4, 8), (192, 64, 30, 64), (256, 16, 2, 5)])
def test_many_tokens_in_groups(E, groups, topk_groups, topk, score, dtype):
    logits = normal(2049, E, dtype, E + groups)
    for group_top in (1, 2):
        for bias in (None, bias_of(E)):
            check_some(logits, topk, bias=bias, score=score, groups=groups, topk_groups=topk_groups, group_top=group_top)


@DTYPES
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(24, 1), (128, 1), (256, 1), (64, 8), (120, 6)])
def test_many_tokens_of_which_some_have_no_scores(E, groups, score, dtype):
    """NaN, +inf and -inf rows and few-expert rows at each of a wave's four places, beside live ones."""
    T = 2055
    logits = normal(T, E, dtype, E)
    inf, nan = float("inf"), float("nan")
    for i in range(4):  # each at every place in a wave of four
        for n, one in enumerate((nan, inf, -inf)):
            logits[100 * n + 5 * i, (7 * i + n) % E] = one
        logits[400 + 5 * i] = -inf
        logits[500 + 5 * i, 1:] = -inf
        logits[600 + 5 * i, ::2] = -inf
        logits[700 + 5 * i] = nan
    logits[T - 1] = nan
    also = [t for n in range(8) for t in range(100 * n, 100 * n + 20)]
    for kw in (dict(), dict(bias=bias_of(E)), dict(renormalize=False)):
        check_some(logits, 5, also, score=score, groups=groups, topk_groups=max(1, groups // 2), **kw)
        if groups > 1:
            check_some(logits, 5, also, score=score, groups=groups, topk_groups=max(1, groups // 2), group_top=2, **kw)


@DTYPES
@pytest.mark.parametrize("biased", [False, True])
def test_many_tokens_ties(biased, dtype):
    g = torch.Generator().manual_seed(5)
    logits = torch.randint(-1, 2, (2053, 96), generator=g).to(dtype).cuda()
    bias = torch.full((96,), 0.25).cuda() if biased else None
    for score in ("softmax", "sigmoid"):
        check_some(logits, 20, bias=bias, score=score)
        for top in (1, 2):
            check_some(logits, 6, bias=bias, score=score, groups=6, topk_groups=2, group_top=top)


@DTYPES
@pytest.mark.parametrize("E,start,wide", [(64, 0, 67), (64, 3, 80), (128, 8, 160), (60, 1, 61), (256, 5, 300)])
def test_many_tokens_strided(E, start, wide, dtype):
    """Rows that begin on any element, with wide loads and without."""
    logits = normal(2051, wide, dtype, wide)
    check_some(logits[:, start:start + E], 6)
    check_some(logits[:, start:start + E], 6, bias=bias_of(E), score="sigmoid")
