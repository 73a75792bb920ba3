"""awq_gemm_fused against its formula in float64 (weights from the oracle's dequantisation).

Tolerances, elementwise, from the arithmetic.  u = 2^-24, q half a step of the activations' type,
tiny half its smallest step.
  P = x . W is a sum of exact terms in fp32, its running value multiplied by a quotient of scales at
    each of the G group boundaries (three roundings, one a reciprocal good to two of u), over at
    most 32 splits and 8 waves: off by dP = (K + 4 G + 48) u A, A = sum |x| |W|.
  v = P + bias: dv = dP + u |v|.
  f(v): |f'| <= 1.13, so 1.13 dv, and its own arithmetic: silu's exponent carries u |v|, that of
    gelu_tanh 14 u |w| (w its polynomial, formed by five roundings); gelu's erfc is good to 16 steps
    and its argument's rounding counts v^2 times: |f| (40 u + u |v|, 14 u |w| or 6 u v^2), and what is
    below fp32's normal range may be flushed: 2^-126 |v|.
  gated: |up| df + |f| dup + df dup + u |f up|;  y: |scale| times that + 3 u (|residual| + |scale f|),
    then q |y| + tiny.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import w4a16_weight_only_amd as awq
from oracle import awq_ref as oracle
from tests.fused_sizes import GATED_TILES, TILES
from w4a16_weight_only_amd import synth

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
ACTS = [None, "relu", "silu", "gelu", "gelu_tanh"]
TYPES = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a HIP GPU")
    awq.load_library()


class Weight:
    def __init__(self, K, C, g, seed, edit=None):
        rng = np.random.default_rng(seed)
        self.G = 1 if g == -1 else K // g
        self.g = g
        self.qw, self.qz = synth.random_words(rng, (K, C // 8)), synth.random_words(rng, (self.G, C // 8))
        self.sc = (rng.uniform(0.5, 1.5, (self.G, C)) / (6.5 * np.sqrt(K))).astype(np.float16)
        if edit is not None:
            edit(self)
        self.dev = tuple(torch.from_numpy(a).cuda() for a in (self.qw, self.qz, self.sc))
        self.W = torch.from_numpy(oracle.dequant_ref(self.qw, self.qz, self.sc, g)).cuda().double()


def f_of(kind, v, dv):
    """f(v) and how far it is off for v off by dv."""
    if kind is None:
        return v, dv
    if kind == "relu":
        return v.clamp_min(0.0), dv
    own = 40 * U
    if kind == "silu":
        f = v * torch.sigmoid(v)
        own = own + U * v.abs()
    elif kind == "gelu":
        f = v * torch.special.ndtr(v)
        own = own + 6 * U * v * v
    else:
        w = math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)
        f = v * torch.sigmoid(2.0 * w)
        own = own + 14 * U * w.abs()
    return f, 1.13 * dv + f.abs() * own + 2.0 ** -126 * v.abs()


def expected(x, w, bias, act, gated, residual, scale):
    X = x.double().reshape(-1, x.shape[-1])
    P = X @ w.W
    dv = (X.shape[1] + 4 * w.G + 48) * U * (X.abs() @ w.W.abs())
    if bias is not None:
        P = P + bias.double()
        dv = dv + U * P.abs()
    if gated:
        N = P.shape[1] // 2
        f, df = f_of(act, P[:, :N], dv[:, :N])
        up, dup = P[:, N:], dv[:, N:]
        df = up.abs() * df + f.abs() * dup + df * dup + U * (f * up).abs()
        f = f * up
    else:
        f, df = f_of(act, P, dv)
    y = scale * f
    dy = abs(scale) * df
    if residual is not None:
        r = residual.double().reshape(y.shape)
        dy = dy + 3 * U * (r.abs() + y.abs())
        y = y + r
    else:
        dy = dy + U * y.abs()
    return y, dy


def close(got, y, dy, where):
    allow = dy + HALF[got.dtype] * y.abs() + TINY[got.dtype]
    off = (got.double().reshape(y.shape) - y).abs()
    bad = ~(off <= allow)
    assert not bad.any(), f"{where}: {int(bad.sum())} of {bad.numel()}, worst {float((off / allow).max()):.3g}"


def rand(gen, *shape, dtype, size=1.0):
    return (size * torch.randn(shape, device="cuda", generator=gen)).to(dtype)


def check(M, K, N, g, dtype, act=None, gated=False, bias=False, residual=False, scale=1.0, seed=0, w=None):
    gen = torch.Generator(device="cuda").manual_seed(seed + M)
    C = 2 * N if gated else N
    w = w or Weight(K, C, g, seed + K + N)
    x = rand(gen, M, K, dtype=dtype)
    b = rand(gen, C, dtype=dtype) if bias else None
    r = rand(gen, M, N, dtype=dtype) if residual else None
    where = f"{M} x {K} -> {N} g {g} {dtype} {act} gated {gated} bias {bias} residual {residual}"
    print(where, flush=True)
    y = awq.awq_gemm_fused(x, *w.dev, b, g, activation=act, gated=gated, residual=r, scale=scale)
    assert y.dtype == dtype and y.shape == (M, N)
    close(y, *expected(x, w, b, act, gated, r, scale), where)
    return y


STREAM = [(1, 32, 32, 32), (1, 4096, 4096, 128), (2, 96, 288, 32), (3, 2048, 1408, -1), (4, 1024, 96, 64),
          (5, 192, 512, 64), (8, 4096, 2048, 128), (9, 512, 544, 32), (16, 11008, 256, 64), (17, 1024, 1024, 128),
          (33, 2048, 320, -1), (64, 4096, 1408, 128), (72, 64, 4096, 32), (73, 320, 544, 64), (200, 2048, 1024, 64),
          (500, 1408, 2048, 128)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,N,g", STREAM)
def test_few_rows(M, K, N, g, dtype):
    for i, gated in enumerate((False, True)):
        w = Weight(K, 2 * N if gated else N, g, M + K)
        check(M, K, N, g, dtype, gated=gated, w=w)
        check(M, K, N, g, dtype, ACTS[(M + i) % 5], gated, True, True, 0.5, w=w)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,N,g", sum(TILES.values(), []))
def test_row_tiles(M, K, N, g, dtype):
    w = Weight(K, N, g, M + K)
    check(M, K, N, g, dtype, w=w)
    check(M, K, N, g, dtype, ACTS[M % 5], False, True, True, 0.5, w=w)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,N,g", sum(GATED_TILES.values(), []))
def test_gated_row_tiles(M, K, N, g, dtype):
    w = Weight(K, 2 * N, g, M + K)
    check(M, K, N, g, dtype, "silu", True, w=w)
    check(M, K, N, g, dtype, ACTS[M % 5], True, True, True, 2.0, w=w)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,K,N", [(7, 256, 288), (75, 320, 22016)])
def test_activations(M, K, N, gated, act):
    """Every activation with and without each of its companions; values from far below to far above 0."""
    w = Weight(K, 2 * N if gated else N, 64, 5, edit=lambda w: w.sc.__imul__(np.float16(6.0)))
    for bias in (False, True):
        for residual in (False, True):
            check(M, K, N, 64, torch.float16, act, gated, bias, residual, -1.5, w=w)


@pytest.mark.parametrize("M", [3, 40, 300])
def test_scales_of_zero_and_negative(M):
    def edit(w):
        w.sc[0, ::3] = 0.0
        w.sc[-1, 1::5] = 0.0
        w.sc[:, 7] = 0.0
        w.sc[1, ::2] *= -1
    for dtype in TYPES:
        check(M, 256, 22528 if M == 300 else 544, 64, dtype, "silu", False, True, True,
              w=Weight(256, 22528 if M == 300 else 544, 64, 9, edit))


def test_exact_integers():
    """x of ones and scales of one: sums of integers, which come out exactly."""
    K, N = 512, 1056
    w = Weight(K, N, 128, 3, edit=lambda w: w.sc.__imul__(np.float16(0.0)).__iadd__(np.float16(1.0)))
    for M in (1, 6, 30):
        x = torch.ones(M, K, dtype=torch.float16, device="cuda")
        y = awq.awq_gemm_fused(x, *w.dev, None, 128)
        assert torch.equal(y.double(), (x.double() @ w.W).half().double())


@pytest.mark.parametrize("M,N", [(6, 544), (50, 544), (300, 22528)])
@pytest.mark.parametrize("dtype", TYPES)
def test_special_values_stay_in_their_row(M, N, dtype):
    w = Weight(256, N, 64, 4)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, r = rand(gen, M, 256, dtype=dtype), rand(gen, M, N, dtype=dtype)
    clean = awq.awq_gemm_fused(x, *w.dev, None, 64, activation="relu", residual=r)
    x[1, 100], x[3, 5] = float("nan"), float("inf")
    r[4, 9] = float("nan")
    y = awq.awq_gemm_fused(x, *w.dev, None, 64, activation="relu", residual=r)
    assert torch.isnan(y[1]).all()
    want = x[3].double() @ w.W  # infinite, or NaN where the weight is zero
    assert torch.equal(torch.isposinf(want), torch.isposinf(y[3])) and torch.equal(torch.isnan(want), torch.isnan(y[3]))
    clean[4, 9] = float("nan")
    for row in [0, 2, 4] + list(range(5, M)):
        assert torch.equal(torch.nan_to_num(y[row], nan=7.0), torch.nan_to_num(clean[row], nan=7.0))


@pytest.mark.parametrize("M,N", [(1, 4096), (19, 1408), (300, 22528)])
def test_in_place_and_leading_dimensions(M, N):
    w = Weight(512, N, 128, 8)
    gen = torch.Generator(device="cuda").manual_seed(2)
    x, r = rand(gen, M, 512, dtype=torch.bfloat16), rand(gen, M, N, dtype=torch.bfloat16)
    y = awq.awq_gemm_fused(x, *w.dev, residual=r)
    y1 = awq.awq_gemm_fused(x.view(1, M, 1, 512), *w.dev, residual=r.view(1, M, 1, N))
    assert y1.shape == (1, M, 1, N) and torch.equal(y1.view(M, N), y)
    again = awq.awq_gemm_fused(x, *w.dev, residual=r, out=r)
    assert again is r and torch.equal(r, y)


def test_same_bits_every_time():
    w = Weight(4096, 2048, 128, 8)
    for M in (1, 8, 30):
        x = rand(torch.Generator(device="cuda").manual_seed(M), M, 4096, dtype=torch.float16)
        first = awq.awq_gemm_fused(x, *w.dev)
        for _ in range(20):
            assert torch.equal(awq.awq_gemm_fused(x, *w.dev), first)


def test_graphs_side_by_side():
    """Two graphs captured on one stream, replayed on two others at once, with eager calls between."""
    w = Weight(4096, 1024, 128, 8)
    gen = torch.Generator(device="cuda").manual_seed(3)
    xs = [rand(gen, m, 4096, dtype=torch.float16) for m in (1, 20)]
    graphs, ys = [], []
    for x in xs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(4):
                y = awq.awq_gemm_fused(x, *w.dev, activation="gelu")
        graphs.append(graph)
        ys.append(y)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for k in range(5):
        for x in xs:
            x.add_(0.25 * k)
        want = [awq.awq_gemm_fused(x, *w.dev, activation="gelu") for x in xs]
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                for _ in range(3):
                    graph.replay()
        torch.cuda.synchronize()
        for y, wanted in zip(ys, want):
            assert torch.equal(y, wanted)


def test_streams_at_once():
    w = Weight(4096, 1024, 128, 8)
    x = rand(torch.Generator(device="cuda").manual_seed(3), 2, 4096, dtype=torch.float16)
    want = awq.awq_gemm_fused(x, *w.dev)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(10):
        for stream in streams:
            with torch.cuda.stream(stream):
                got.append(awq.awq_gemm_fused(x, *w.dev))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in got)


def test_empty_and_refusals():
    w = Weight(256, 512, 64, 1)
    x = torch.zeros(4, 256, dtype=torch.float16, device="cuda")
    y = torch.zeros(4, 512, dtype=torch.float16, device="cuda")
    assert awq.awq_gemm_fused(x[:0], *w.dev, group_size=64).shape == (0, 512)
    qw, qz, sc = w.dev
    call = lambda *a, **k: awq.awq_gemm_fused(*a, group_size=k.pop("group_size", 64), **k)  # noqa: E731
    wide = torch.zeros(4, 1024, dtype=torch.float16, device="cuda")
    for error, bad in [
        (TypeError, lambda: call(x.float(), *w.dev)),
        (TypeError, lambda: call(x, qw.long(), qz, sc)),
        (TypeError, lambda: call(x, qw, qz, sc.bfloat16())),
        (TypeError, lambda: call(x, *w.dev, y[0].bfloat16())),
        (ValueError, lambda: call(x, *w.dev, y[0, :256])),
        (ValueError, lambda: call(x[:, :128].contiguous(), *w.dev)),
        (ValueError, lambda: call(x, *w.dev, group_size=96)),
        (ValueError, lambda: call(x, *w.dev, group_size=16)),
        (ValueError, lambda: call(x, *w.dev, group_size=0)),
        (ValueError, lambda: call(x, *w.dev, group_size=32)),
        (ValueError, lambda: call(x, *w.dev, activation="tanh")),
        (ValueError, lambda: call(x.t(), *w.dev)),
        (ValueError, lambda: call(x.cpu(), *w.dev)),
        (ValueError, lambda: call(x, *w.dev, residual=y[:2])),
        (TypeError, lambda: call(x, *w.dev, residual=y.bfloat16())),
        (ValueError, lambda: call(x, *w.dev, gated=True, residual=y)),
        (ValueError, lambda: call(x, *w.dev, out=y[:, :256])),
        (ValueError, lambda: call(x, *w.dev, residual=wide.view(-1)[:2048].view(4, 512),
                                  out=wide.view(-1)[512:2560].view(4, 512))),
        (ValueError, lambda: call(wide.view(-1)[:1024].view(4, 256), *w.dev, out=wide.view(-1)[:2048].view(4, 512))),
    ]:
        with pytest.raises(error):
            bad()
