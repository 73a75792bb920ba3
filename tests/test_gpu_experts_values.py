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


@DTYPES
@pytest.mark.parametrize("T", [1, 5, 40, 300])
def test_layer_module_keeps_nan(T, dtype):
    """A token without scores (a NaN in x, router products that overflow to infinity) comes out as
    NaN; every other token's bits are those of a clean call, a token without experts' zeros too."""
    E, topk, K, inner, g = 16, 4, 256, 128, 64
    up, down = Layer(E, K, 2 * inner, g, 21), Layer(E, inner, K, g, 22)
    router = activations((E, K), dtype, 23) / 16
    layer = awq.AwqMoe(router, up.dev, down.dev, topk, g)
    x = activations((T, K), dtype, 24)
    clean = layer(x)
    assert torch.isfinite(clean).all()
    for bad in (float("nan"), float("inf"), -float("inf")):
        y = x.clone()
        y[T // 2, 3] = bad
        got = layer(y)
        keep = torch.arange(T) != T // 2
        assert torch.equal(got[keep], clean[keep])
        assert torch.isnan(got[T // 2]).all()
    none = awq.AwqMoe(router, up.dev, down.dev, topk, g, bias=torch.full((E,), -float("inf"), device="cuda"))
    assert (none(x) == 0).all()
    far = torch.finfo(dtype).max
    big = torch.full((T, K), 0.0, dtype=dtype, device="cuda")
    big[T // 2] = far  # finite: it is the logits that are not
    router[:, 0] = far
    assert torch.isnan(layer(big)[T // 2]).all()


@DTYPES
@pytest.mark.parametrize("T,topk", [(1, 2), (3, 5), (40, 3), (300, 2)])
def test_nan_weights_on_request(T, topk, dtype):
    """nan_weights: a token with a NaN weight is NaN also where that slot is not routed; nothing
    else changes, an infinite weight of an unrouted slot adds nothing."""
    E, K, inner, N, g = 4, 64, 96, 64, 32
    up, down = Layer(E, K, 2 * inner, g, 25), Layer(E, inner, N, g, 26)
    x, h = activations((T, K), dtype, 27), activations((T * topk, inner), dtype, 28)
    rng = np.random.default_rng(29)
    ids = torch.from_numpy(rng.integers(-1, E + 1, (T, topk)).astype(np.int32)).cuda()
    w = torch.from_numpy(rng.uniform(0.1, 1, (T, topk)).astype(np.float32)).cuda()
    off = (ids < 0) | (ids >= E)
    w[off] = float("inf")
    calls = [lambda **kw: awq.awq_moe_down(h, *down.dev, ids, w, g, **kw),
             lambda **kw: awq.awq_moe_mlp(x, up.dev, down.dev, ids, w, g, **kw)]
    for call in calls:
        assert torch.equal(call(nan_weights=True), call())
    ids[0, topk - 1], w[0, topk - 1] = E, float("nan")
    for call in calls:
        plain, kept = call(), call(nan_weights=True)
        assert torch.isfinite(plain).all() and torch.isnan(kept[0]).all() and torch.equal(kept[1:], plain[1:])


@DTYPES
@pytest.mark.parametrize("T", [1, 33])
def test_layer_module_of_a_32_bit_router(T, dtype):
    """A router in fp32 gives fp32 logits: experts that 16-bit logits would tie keep their order."""
    E, topk, K, inner, g = 16, 2, 256, 128, 64
    up, down = Layer(E, K, 2 * inner, g, 31), Layer(E, inner, K, g, 32)
    router = torch.zeros(E, K, device="cuda")
    router[:, 0] = 1.0 + 2.0 ** -14 * torch.arange(E, device="cuda")  # one value in 16 bits
    x = activations((T, K), dtype, 33)
    x[:, 0] = 1.0
    y = awq.AwqMoe(router, up.dev, down.dev, topk, g)(x)
    assert y.dtype == dtype
    w, ids = awq.awq_moe_route(router[:, 0].repeat(T, 1), topk)
    assert ids.cpu().tolist() == [[E - 1, E - 2]] * T
    assert torch.equal(y, awq.awq_moe_mlp(x, up.dev, down.dev, ids, w, g))
    with pytest.raises(TypeError):
        awq.AwqMoe(router.double(), up.dev, down.dev, topk, g)(x)
    with pytest.raises(TypeError):
        awq.AwqMoe(router.to(torch.float16 if dtype is torch.bfloat16 else torch.bfloat16), up.dev, down.dev, topk, g)(x)


@DTYPES
@pytest.mark.parametrize("counts,K,N", [((1,), 4096, 512), ((5, 3), 4096, 512), ((30, 34), 2048, 320),
                                        ((100, 140), 4096, 512), ((300, 190, 100, 230), 1024, 8768)],
                         ids=["1", "8", "64", "240", "tiles"])
def test_equal_scales_in_all_groups_change_nothing(counts, K, N, dtype):
    """Groups of 32 that all have a column's one scale and zero are one group of K: sums of whole
    numbers below 2^24 are exact, and stay so at every boundary, so both give the same bits."""
    E, T = len(counts), sum(counts)
    assert 3 * 15 * K < 2 ** 24
    print(f"equal scales counts={counts} K={K} N={N} {dtype}", flush=True)
    ids, w = routed_by_counts(counts, 12)
    w.fill_(1.0)
    x = torch.from_numpy(np.random.default_rng(13).integers(-3, 4, (T, K)).astype(np.float64)).to(dtype).cuda()

    def same(layer):
        layer.qz[:], layer.sc[:] = layer.qz[:, :1], layer.sc[:, :1]

    many = Layer(E, K, N, 32, 14, same)
    one = (many.dev[0], many.dev[1][:, :1].contiguous(), many.dev[2][:, :1].contiguous())
    assert torch.equal(awq.awq_moe_down(x, *many.dev, ids, w, 32), awq.awq_moe_down(x, *one, ids, w, -1))
    assert torch.equal(awq.awq_moe_gate_up(x, *(t.contiguous() for t in many.dev), ids, 32),
                       awq.awq_moe_gate_up(x, *one, ids, -1))


@DTYPES
@pytest.mark.parametrize("counts", [(3, 2), (100, 140)], ids=["5", "240"])
def test_outputs_over_inputs(counts, dtype):
    """y may lie where h or x was; h may not lie where x is."""
    E, T, K, g = len(counts), sum(counts), 128, 32
    ids, w = routed_by_counts(counts, 41)
    up, down = Layer(E, K, 2 * K, g, 42), Layer(E, K, K, g, 43)
    x = activations((T, K), dtype, 44)
    with pytest.raises(ValueError):
        awq.awq_moe_gate_up(x, *up.dev, ids, g, out=x)
    for call in (lambda v, **kw: awq.awq_moe_down(v, *down.dev, ids, w, g, **kw),
                 lambda v, **kw: awq.awq_moe_mlp(v, up.dev, down.dev, ids, w, g, **kw)):
        want, over = call(x), x.clone()
        assert torch.equal(call(over, out=over), want)
