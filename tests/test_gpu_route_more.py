"""awq_moe_route where scores of different logits round to the same number.

Same comparison and tolerances as test_gpu_route.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import w4a16_weight_only_amd as awq
from tests.test_gpu_route import check, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a HIP GPU")
    awq.load_library()


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
    _, ids = check(logits, topk, score=score, groups=groups, topk_groups=topk_groups, group_top=2)
    want = np.argsort(-logits.cpu().numpy(), axis=1, kind="stable")[:, :topk]
    assert np.array_equal(ids.cpu().numpy(), want)
