"""Values that the routed-expert products have to give exactly: infinities and NaN as IEEE sums of
exact products give them.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import w4a16_weight_only_amd as awq
from tests.test_gpu_experts import Layer, activations, f64, routed_by_counts

pytestmark = pytest.mark.gpu

DTYPES = pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a HIP GPU")
    awq.load_library()


# Slots per expert and columns: ranked and tabled streaming with 4, 8, 16 and 32 rows kept, row
# tiles of three heights.
COUNTS = [((3, 1), 96), ((5, 3), 96), ((9, 8), 288), ((20, 13), 96), ((100, 40), 160), ((300, 190, 100, 230), 8736)]


@DTYPES
@pytest.mark.parametrize("counts,N", COUNTS, ids=[str(sum(c)) for c, _ in COUNTS])
def test_infinities_keep_their_sign(counts, N, dtype):
    """An infinite x makes a product infinite with the sign of its weight, and NaN only where that
    weight is zero (inf * 0); the activation's own formula does the rest."""
    E, T, K, g = len(counts), sum(counts), 160, 32
    print(f"infinities counts={counts} N={N} {dtype}", flush=True)
    ids, w = routed_by_counts(counts, 1)
    w.fill_(1.0)
    up, down = Layer(E, K, 2 * N, g, 2), Layer(E, K, N, g, 3)
    x = activations((T, K), dtype, 4)
    clean = awq.awq_moe_down(x, *down.dev, ids, w, g)
    for t, at, bad in ((0, 0, np.inf), (1, K - 1, -np.inf), (T - 1, 37, np.inf)):
        x[t, at] = bad
    h = f64(awq.awq_moe_gate_up(x, *up.dev, ids, g))
    y = awq.awq_moe_down(x, *down.dev, ids, w, g)
    for t, at, bad in ((0, 0, np.inf), (1, K - 1, -np.inf), (T - 1, 37, np.inf)):
        e = int(ids[t, 0])
        with np.errstate(invalid="ignore", over="ignore"):
            v = bad * down.W[e][at]
            gate, lin = np.split(bad * up.W[e][at], 2)
            ref = gate / (1 + np.exp(-gate)) * lin
        assert np.isinf(v).sum() > 0.8 * N and np.isnan(v).any()
        np.testing.assert_array_equal(f64(y)[t], v)
        np.testing.assert_array_equal(h[t], ref)
    keep = np.setdiff1d(np.arange(T), [0, 1, T - 1])
    assert torch.equal(y[keep], clean[keep])
