"""The routed-expert products at the heights where row tiles change, and the whole MLP where either
product, or both, run on row tiles.  Tolerances as in test_gpu_experts.py; which kernel a size
reaches is checked on the CPU (test_experts_choice.py)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import w4a16_weight_only_amd as awq
from tests.expert_sizes import FAMILIES, HEIGHT_INNER, HEIGHT_KS, HEIGHT_N, HEIGHTS
from tests.test_gpu_experts import Layer, activations, close, down_ref, gate_up_ref, routed_by_counts, routing

pytestmark = pytest.mark.gpu

DTYPES = pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a HIP GPU")
    awq.load_library()


@DTYPES
@pytest.mark.parametrize("K,g", HEIGHT_KS)
@pytest.mark.parametrize("counts", HEIGHTS, ids=["whole", "one off", "two entries"])
def test_heights(counts, K, g, dtype):
    E, T = len(counts), sum(counts)
    print(f"heights counts={counts} K={K} g={g} {dtype}", flush=True)
    ids, w = routed_by_counts(counts, K)
    x = activations((T, K), dtype, K + 1)
    up, down = Layer(E, K, 2 * HEIGHT_INNER, g, 3), Layer(E, K, HEIGHT_N, g, 4)
    close(awq.awq_moe_gate_up(x, *up.dev, ids, g), *gate_up_ref(x, up, ids, dtype), "gate_up")
    close(awq.awq_moe_down(x, *down.dev, ids, w, g), *down_ref(x, down, ids, w, dtype), "down")


@DTYPES
@pytest.mark.parametrize("size,up_streams,down_streams", FAMILIES)
def test_whole_mlp(size, up_streams, down_streams, dtype):
    """The bits of its two halves, which are right; with slots that are not routed and an expert
    twice in a token, and with NaN and infinities in two tokens, which no other token notices."""
    T, E, topk, K, inner, N, g = size
    print(f"mlp {size} {dtype}", flush=True)
    up, down = Layer(E, K, 2 * inner, g, 5), Layer(E, inner, N, g, 6)
    x = activations((T, K), dtype, 7)
    ids, w = routing(T, E, topk, 8)
    ids[::7, 0], ids[3], ids[5] = -1, torch.tensor([E, -9]), torch.tensor([2, 2])
    w[3] = float("nan")
    live = ((ids >= 0) & (ids < E)).flatten()
    h = torch.full((T * topk, inner), 7.0, dtype=dtype, device="cuda")
    awq.awq_moe_gate_up(x, *up.dev, ids, g, out=h)
    assert (h[~live] == 7.0).all() and torch.equal(h[10], h[11])
    ref, tol = gate_up_ref(x, up, ids, dtype)
    m = live.cpu().numpy()
    close(h[live], ref[m], tol[m], "gate_up")
    steps = awq.awq_moe_down(h, *down.dev, ids, w, g)
    close(steps, *down_ref(h, down, ids, w, dtype), "down")
    y = awq.awq_moe_mlp(x, up.dev, down.dev, ids, w, g)
    assert torch.equal(y, steps) and (y[3] == 0).all()
    bad = x.clone()
    bad[1, K - 1], bad[T - 1, 0] = float("inf"), float("nan")
    got = awq.awq_moe_mlp(bad, up.dev, down.dev, ids, w, g)
    keep = np.setdiff1d(np.arange(T), [1, T - 1])
    assert torch.equal(got[keep], y[keep])
    assert not torch.isfinite(got[1]).all() and torch.isnan(got[T - 1]).all()
