"""AwqLinear, AwqMlp and AwqMoe with the operators around the products, alone and in a decoder's order.

The modules run the same calls as the functions (tested against float64 in test_gpu_norm.py,
test_gpu_fused.py and test_gpu_layer.py), so they give their bits.  A chain of blocks is held to
float64 by its 2-norm: every tensor that is rounded on the way is off by at most q (half a step)
of its own 2-norm.  A block rounds its norm, its activations, its product or h, and its output, and its
matrices pass an error's 2-norm on, relative to the value's, at most 4 fold here (random matrices:
their largest singular value over their root mean square one is below 2.5 for these shapes, the
gate's derivative counts at most 1.1 + 1).  4 roundings of q through a factor 4, added to a stream
that is not smaller than the block's output: 16 q a block.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import w4a16_weight_only_amd as awq
from oracle import awq_ref as oracle
from tests.test_gpu_experts import HALF, Layer, f64
from tests.test_gpu_fused import Weight

pytestmark = pytest.mark.gpu

TYPES = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a HIP GPU")
    awq.load_library()


def rand(*shape, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, device="cuda", generator=gen).to(dtype)


@pytest.mark.parametrize("dtype", TYPES)
def test_linear(dtype):
    w = Weight(256, 544, 64, 1)
    x, b, r = rand(3, 2, 256, dtype=dtype, seed=1), rand(544, dtype=dtype, seed=2), rand(3, 2, 544, dtype=dtype, seed=3)
    plain = awq.AwqLinear(*w.dev, b, 64)
    assert torch.equal(plain(x), awq.awq_gemm(x, *w.dev, b, 64))
    assert torch.equal(plain(x, residual=r), awq.awq_gemm_fused(x, *w.dev, b, 64, residual=r))
    assert torch.equal(awq.AwqLinear(*w.dev, b, 64, activation="gelu")(x.transpose(0, 1)),
                       awq.awq_gemm_fused(x.transpose(0, 1).contiguous(), *w.dev, b, 64, activation="gelu"))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [1, 6, 150])
def test_mlp(T, dtype):
    K, inner = 256, 352
    up, down = Weight(K, 2 * inner, 32, 4), Weight(inner, K, 32, 5)
    x = rand(T, 1, K, dtype=dtype, seed=T)
    n, p, t = (rand(K, dtype=dtype, seed=s) for s in (6, 7, 8))
    b = rand(2 * inner, dtype=dtype, seed=9)
    h = awq.awq_norm(x, n)
    z = awq.awq_gemm_fused(h, *up.dev, b, 32, activation="silu", gated=True)
    plain = awq.AwqMlp(up.dev, down.dev, 32, norm=n, up_bias=b, scale=0.5)
    want = awq.awq_gemm_fused(z, *down.dev, None, 32, residual=x, scale=0.5)
    assert torch.equal(plain(x), want)
    assert torch.equal(plain(x, normed=h), want)
    d = awq.awq_gemm_fused(z, *down.dev, None, 32)
    both = plain(x, then=t)
    assert all(torch.equal(a, c) for a, c in zip(both, awq.awq_add_norm(d, x, t, scale=0.5)))
    sandwich = awq.AwqMlp(up.dev, down.dev, 32, norm=n, up_bias=b, post_norm=p)
    y, r = awq.awq_add_norm(d, x, None, post_weight=p)
    assert y is None and torch.equal(sandwich(x), r)
    assert torch.equal(sandwich(x, then=t)[1], r)
    ungated = awq.AwqMlp(tuple(w[:, :inner // 8].contiguous() if w.dtype == torch.int32 else w[:, :inner].contiguous()
                               for w in up.dev), down.dev, 32, activation="gelu_tanh", gated=False)
    assert ungated(x).shape == x.shape


@pytest.mark.parametrize("dtype", TYPES)
def test_moe_in_one_call(dtype):
    E, topk, K, inner, g = 16, 4, 256, 128, 64
    up, down = Layer(E, K, 2 * inner, g, 1), Layer(E, inner, K, g, 2)
    for router_type in (dtype, torch.float32):
        router = rand(E, K, dtype=router_type, seed=3) / 8
        layer = awq.AwqMoe(router, up.dev, down.dev, topk, g, one_call=True, score="sigmoid")
        parts = awq.AwqMoe(router, up.dev, down.dev, topk, g, score="sigmoid")
        for T in (1, 16):
            x, r = rand(T, 1, K, dtype=dtype, seed=T), rand(T, 1, K, dtype=dtype, seed=T + 1)
            want = awq.awq_moe_layer(x[:, 0].contiguous(), router, up.dev, down.dev, topk, g, score="sigmoid",
                                     round_logits=router_type is dtype, residual=r[:, 0].contiguous())
            got = layer(x, residual=r)
            assert got.shape == x.shape and torch.equal(got[:, 0], want)
            assert float((layer(x) - parts(x)).double().norm()) <= 2 * HALF[dtype] * float(parts(x).double().norm())
        x = rand(17, 1, K, dtype=dtype, seed=17)  # 68 slots: the calls of the default
        assert torch.equal(layer(x), parts(x))
        assert torch.equal(layer(x, residual=x), x + parts(x))
        with pytest.raises(ValueError):
            layer(x, residual=x[:4])
        for module in (layer, parts):
            assert module(x[:0], residual=x[:0]).shape == (0, 1, K)


@pytest.mark.parametrize("dtype", TYPES)
def test_moe_residuals_whatever_the_token_count(dtype):
    """16 tokens take one call, 17 the calls of the default: both take a residual in fp32 (and give fp32), one
    that begins on its element's alignment only, one with its columns apart; the one call such a router too."""
    E, topk, K, inner, g = 16, 4, 256, 128, 64
    up, down = Layer(E, K, 2 * inner, g, 1), Layer(E, inner, K, g, 2)
    router = rand(E, K, dtype=dtype, seed=3) / 8
    layer = awq.AwqMoe(router, up.dev, down.dev, topk, g, one_call=True)
    apart = rand(K, E, dtype=dtype, seed=3).t()
    apart.copy_(router)
    odd = torch.empty(E * K + 1, dtype=dtype, device="cuda")[1:].view(E, K)
    odd.copy_(router)
    for T in (16, 17):
        x, r = rand(T, K, dtype=dtype, seed=T), rand(T, K, dtype=torch.float32, seed=T + 1)
        y = layer(x)
        got = layer(x, residual=r)
        assert got.dtype == torch.float32 and torch.equal(got, r + y)
        want = layer(x, residual=r.to(dtype))
        off = torch.empty(T * K + 1, dtype=dtype, device="cuda")[1:].view(T, K)
        off.copy_(r)
        assert torch.equal(layer(x, residual=off), want)
        assert torch.equal(layer(x, residual=r.to(dtype).t().contiguous().t()), want)
        for same in (apart, odd) if T == 16 else ():
            other = awq.AwqMoe(same, up.dev, down.dev, topk, g, one_call=True)
            assert torch.equal(other(x, residual=r.to(dtype)), want)


def float64_chain(x, norms, dense, moe):
    """Two dense blocks around a routed one, in float64."""
    def rms(v, w):
        return v / np.sqrt((v * v).mean(axis=1, keepdims=True) + 1e-6) * w

    def mlp(v, up, down):
        p = v @ up.W.cpu().numpy()
        a, b = np.split(p, 2, axis=1)
        return (a / (1 + np.exp(-a)) * b) @ down.W.cpu().numpy()

    r = f64(x)
    n = [f64(w) for w in norms]
    r = r + mlp(rms(r, n[0]), *dense[0])
    router, up, down, topk = moe
    v = rms(r, n[1])
    weights, ids = oracle.route_ref(v @ f64(router).T, topk)
    for t in range(len(r)):
        for w, e in zip(weights[t], ids[t]):
            p = v[t] @ up.W[e]
            a, b = np.split(p, 2)
            r[t] += w * ((a / (1 + np.exp(-a)) * b) @ down.W[e])
    r = r + rms(mlp(rms(r, n[2]), *dense[1]), n[3])
    return r


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [1, 8])
def test_chain_eager_and_captured(T, dtype):
    """norm, dense block, norm and routed block, sandwich block: against float64, then captured and
    replayed several times with other inputs and eager calls between."""
    K, inner, E, topk, g = 512, 704, 16, 4, 64
    dense = [(Weight(K, 2 * inner, g, s), Weight(inner, K, g, s + 1)) for s in (1, 3)]
    up, down = Layer(E, K, 2 * inner, g, 5), Layer(E, inner, K, g, 6)
    norms = [(1 + 0.1 * rand(K, dtype=torch.float32, seed=s)).to(dtype) for s in range(4)]
    # A router whose choices are far apart: experts read a coordinate each, amplified.
    router = torch.zeros(E, K, device="cuda")
    router[torch.arange(E), 7 * torch.arange(E)] = 8.0
    x = rand(T, K, dtype=dtype, seed=11)
    first = awq.AwqMlp(*(w.dev for w in dense[0]), g, norm=norms[0])
    layer = awq.AwqMoe(router, up.dev, down.dev, topk, g, one_call=True)
    last = awq.AwqMlp(*(w.dev for w in dense[1]), g, norm=norms[2], post_norm=norms[3])

    def run():
        normed, r = first(x, then=norms[1])
        return last(layer(normed, residual=r))

    y = run()
    want = float64_chain(x, norms, dense, (router, up, down, topk))
    assert np.linalg.norm(f64(y) - want) <= 3 * 16 * HALF[dtype] * np.linalg.norm(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run()
    for k in range(4):
        x.copy_(rand(T, K, dtype=dtype, seed=20 + k))
        eager = run()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(captured, eager)
