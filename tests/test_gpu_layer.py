"""awq_moe_layer against the oracle's routing and the formulas in float64.

x and the router hold small multiples of powers of two, so that the logits are exact in fp32 (and tie
now and then, which goes to the lowest index): the choice of experts is the oracle's.
Tolerance: that of the whole MLP with h in two terms (test_gpu_experts.py), before its rounding; the
weights, fp32 quotients of a few exponentials, carry 16 u of themselves, the sum over slots and
splits (topk + 34) u of its terms, the residual 2 u (|residual| + |y|); y is rounded once.
"""
from __future__ import annotations

import threading

import numpy as np
import pytest
import torch

import w4a16_weight_only_amd as awq
from oracle import awq_ref as oracle
from tests.test_gpu_experts import HALF, TINY, U, Layer, f64, gate_up_ref, product

pytestmark = pytest.mark.gpu

TYPES = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a HIP GPU")
    awq.load_library()


class Case:
    def __init__(self, T, E, K, inner, N, g, dtype, router_type, seed, residual=True, edit=None):
        rng = np.random.default_rng(seed)
        self.g, self.dtype = g, dtype
        self.up, self.down = Layer(E, K, 2 * inner, g, seed + 1), Layer(E, inner, N, g, seed + 2)
        # Logits of a spread of about 1.5, in steps of 2^-7 or coarser.
        step = 2.0 ** -min(6, int(np.log2(np.sqrt(K) * 2)))
        x = rng.integers(-4, 5, (T, K)) / 2.0
        router = rng.integers(-2, 3, (E, K)) * step / 2.0
        if edit is not None:
            edit(x, router)
        self.x = torch.from_numpy(x).to(dtype).cuda()
        self.router = torch.from_numpy(router).to(router_type).cuda()
        self.residual = torch.from_numpy(rng.standard_normal((T, N))).to(dtype).cuda() if residual else None

    def run(self, topk, **kw):
        return awq.awq_moe_layer(self.x, self.router, self.up.dev, self.down.dev, topk, self.g, residual=self.residual, **kw)

    def check(self, topk, bias=None, round_logits=False, **routing):
        T, N = self.x.shape[0], self.down.W.shape[2]
        logits = f64(self.x) @ f64(self.router).T
        if round_logits:
            logits = f64(torch.from_numpy(logits).to(self.dtype))
        b = None if bias is None else f64(bias)
        weights, ids = oracle.route_ref(logits, topk, bias=b, **routing)
        lost = np.isnan(weights).any(axis=1)
        y = self.run(topk, bias=bias, round_logits=round_logits, **routing)
        assert y.dtype == self.dtype and y.shape == (T, N)
        idt = torch.from_numpy(ids.astype(np.int32))
        r = HALF[self.dtype]
        h, tol = gate_up_ref(self.x, self.up, idt, self.dtype)
        dh = (tol - TINY[self.dtype] - r * np.abs(h)) / (1 + r)
        dh = dh + r * r * (np.abs(h) + dh) + TINY[self.dtype]
        flat = ids.ravel()
        v, d = product(h, self.down, flat, self.dtype)
        A = np.abs(self.down.W)
        for e in range(A.shape[0]):
            m = flat == e
            if m.any():
                d[m] = 2 * d[m] * (1 + 2 * r) + dh[m] @ A[e]
        w = np.where(flat >= 0, weights.ravel(), 0.0)[:, None]
        fold = lambda a: a.reshape(T, topk, -1).sum(axis=1)  # noqa: E731
        want = fold(w * v)
        off = fold(np.abs(w) * d) + (topk + 50) * U * fold(np.abs(w * v))
        if self.residual is not None:
            want = want + f64(self.residual)
            off = off + 2 * U * (np.abs(f64(self.residual)) + np.abs(want))
        off = off + r * (np.abs(want) + off) + TINY[self.dtype]
        got = f64(y)
        assert np.isnan(got[lost]).all()
        bad = ~(np.abs(got - want) <= off)[~lost]
        assert not bad.any(), f"{bad.sum()} of {bad.size}, worst {np.nanmax((np.abs(got - want) / off)[~lost]):.3g}"
        return y, ids


# (T, E, topk, K, inner, N, g)
SIZES = [(1, 4, 2, 32, 32, 32, 32), (1, 64, 8, 2048, 1408, 2048, 128), (2, 8, 2, 4096, 512, 1024, -1),
         (3, 16, 4, 96, 160, 288, 32), (4, 60, 4, 512, 544, 544, 32), (5, 8, 1, 1024, 96, 4096, -1),
         (7, 64, 8, 2048, 1408, 2048, 64), (8, 128, 8, 256, 320, 256, 64), (9, 300, 4, 128, 128, 128, 128),
         (16, 8, 2, 1024, 1536, 1024, 128), (16, 1024, 4, 64, 64, 64, 64), (33, 2, 1, 256, 128, 288, 64),
         (64, 1, 1, 512, 288, 320, 32), (64, 40, 1, 512, 288, 320, 32), (1, 80, 64, 64, 64, 96, 32),
         (32, 2, 2, 320, 96, 64, 32)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_sizes(size, dtype):
    T, E, topk, K, inner, N, g = size
    print(size, dtype, flush=True)
    Case(T, E, K, inner, N, g, dtype, dtype, 3).check(topk)
    Case(T, E, K, inner, N, g, dtype, torch.float32, 4, residual=False).check(topk, score="sigmoid", scale=2.5)


@pytest.mark.parametrize("E,groups,topk_groups", [(16, 4, 2), (60, 4, 3), (128, 8, 4), (512, 16, 3), (7, 7, 5)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_top", [1, 2])
def test_routing(E, groups, topk_groups, score, group_top):
    rng = np.random.default_rng(E)
    bias = torch.from_numpy((rng.integers(-8, 9, E) / 16.0).astype(np.float32)).cuda()
    case = Case(6, E, 128, 64, 96, 64, torch.float16, torch.float32, E)
    for b in (None, bias):
        for renormalize in (True, False):
            case.check(4, bias=b, score=score, groups=groups, topk_groups=topk_groups, group_top=group_top,
                       renormalize=renormalize, scale=1.5)


def test_rounded_logits():
    for dtype in TYPES:
        case = Case(8, 64, 2048, 64, 64, 64, dtype, torch.float32, 5)
        case.check(8, round_logits=True)
        case.check(8)


@pytest.mark.parametrize("dtype", TYPES)
def test_switched_off_and_lost(dtype):
    """Experts switched off by a bias of -inf, tokens without experts, rows that are not finite."""
    bias = torch.zeros(8, device="cuda")
    bias[1:6] = -float("inf")
    case = Case(5, 8, 256, 96, 288, 32, dtype, dtype, 1)
    _, ids = case.check(4, bias=bias)
    assert (ids[:, 3] == -1).all()
    clean = case.run(2)
    none = case.run(2, bias=torch.full((8,), -float("inf"), device="cuda"))
    assert torch.equal(none, case.residual)
    case.residual = None
    assert not case.run(2, bias=torch.full((8,), -float("inf"), device="cuda")).any()
    case = Case(5, 8, 256, 96, 288, 32, dtype, dtype, 1)
    case.x[1, 7] = float("nan")
    case.x[3, 9] = float("inf")
    y = case.run(2)
    assert torch.isnan(y[1]).all() and torch.isnan(y[3]).all()
    for row in (0, 2, 4):
        assert torch.equal(y[row], clean[row])
    case.x.fill_(float("nan"))
    assert torch.isnan(case.run(2)).all()


def test_all_to_one_expert():
    def edit(x, router):
        x[:, 0] = 2.0
        router[5, 0] = 32.0
    for T in (16, 17, 40):
        _, ids = Case(T, 8, 512, 160, 544, 32, torch.bfloat16, torch.float32, T, edit=edit).check(1)
        assert (ids == 5).all()


def test_against_the_parts():
    """The same experts and, within two roundings, the same y as routing and MLP in calls of their own."""
    for dtype in TYPES:
        case = Case(7, 64, 1024, 704, 1024, 64, dtype, torch.float32, 8, residual=False)
        logits = case.x.float() @ case.router.t()
        weights, ids = awq.awq_moe_route(logits, 8)
        want = awq.awq_moe_mlp(case.x, case.up.dev, case.down.dev, ids, weights, 64)
        got = case.run(8)
        assert float((got.double() - want.double()).norm() / want.double().norm()) <= 2 * HALF[dtype]


@pytest.mark.parametrize("dtype", TYPES)
def test_one_token_whose_h_is_long(dtype):
    """So many experts that K of the second product is not split, and more columns of h than one token's form
    keeps: the form of several tokens.  Against routing and MLP in calls of their own, within two roundings."""
    E, topk, K, inner, N, g = 64, 64, 64, 8224, 1024, 32
    gen = torch.Generator(device="cuda").manual_seed(31)
    words = lambda *s: torch.randint(-(1 << 31), 1 << 31, s, dtype=torch.int32, device="cuda", generator=gen)  # noqa: E731

    def packed(rows, cols):
        scales = torch.rand((E, rows // g, cols), device="cuda", generator=gen).add_(0.5).mul_(1 / (6.5 * rows ** 0.5))
        return words(E, rows, cols // 8), words(E, rows // g, cols // 8), scales.half()

    up, down = packed(K, 2 * inner), packed(inner, N)
    x = torch.randn((1, K), device="cuda", generator=gen).to(dtype)
    router = torch.randn((E, K), device="cuda", generator=gen)
    weights, ids = awq.awq_moe_route(x.float() @ router.t(), topk)
    want = awq.awq_moe_mlp(x, up, down, ids, weights, g)
    first = awq.awq_moe_layer(x, router, up, down, topk, g)
    assert float((first.double() - want.double()).norm() / want.double().norm()) <= 2 * HALF[dtype]
    for _ in range(10):
        assert torch.equal(awq.awq_moe_layer(x, router, up, down, topk, g), first)


def test_same_bits_and_in_place():
    case = Case(5, 64, 2048, 1408, 2048, 128, torch.float16, torch.float16, 2)
    first = case.run(8)
    for _ in range(30):
        assert torch.equal(case.run(8), first)
    residual = case.residual.clone()
    assert torch.equal(awq.awq_moe_layer(case.x, case.router, case.up.dev, case.down.dev, 8, 128, residual=residual,
                                         out=residual), first)
    x = case.x.clone()
    assert torch.equal(awq.awq_moe_layer(x, case.router, case.up.dev, case.down.dev, 8, 128, residual=case.residual,
                                         out=x), first)


def test_graphs_side_by_side():
    """Two graphs captured on one stream, replayed on two others at once, with eager calls between."""
    cases = [Case(T, 64, 1024, 704, 1024, 64, torch.float16, torch.float32, T) for T in (1, 6)]
    graphs, ys = [], []
    for case in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(3):
                y = case.run(8)
        graphs.append(graph)
        ys.append(y)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for k in range(5):
        for case in cases:
            case.x.neg_()
        want = [case.run(8) for case in cases]
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                for _ in range(3):
                    graph.replay()
        torch.cuda.synchronize()
        for y, wanted in zip(ys, want):
            assert torch.equal(y, wanted)


def test_streams_at_once():
    cases = [Case(T, 64, 2048, 1408, 2048, 128, torch.bfloat16, torch.bfloat16, T) for T in (1, 8, 3)]
    want = [case.run(8) for case in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for _ in range(10):
        for case, stream in zip(cases, streams):
            with torch.cuda.stream(stream):
                got.append(case.run(8))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i % 3]) for i, y in enumerate(got))


def test_threads_on_one_stream():
    """Two threads' calls on one stream share its scratch; a call's two launches stay together."""
    cases = [Case(4, 16, 256, 128, 256, 64, torch.float16, torch.float32, seed) for seed in (71, 72)]
    want = [c.run(4) for c in cases]
    torch.cuda.synchronize()
    wrong = [-1, -1]

    def calls(i):
        got = [cases[i].run(4) for _ in range(300)]
        torch.cuda.synchronize()
        wrong[i] = sum(not torch.equal(y, want[i]) for y in got)

    threads = [threading.Thread(target=calls, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == [0, 0]


def test_a_layer_beside_a_fused_product_from_two_threads():
    """Calls of several kinds from two threads on one stream: each call's launches may come between those
    of the other thread's, whose scratch they leave alone."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    w = (torch.randint(-(1 << 31), 1 << 31, (4096, 512), dtype=torch.int32, device="cuda", generator=gen),
         torch.randint(-(1 << 31), 1 << 31, (32, 512), dtype=torch.int32, device="cuda", generator=gen),
         torch.rand((32, 4096), device="cuda", generator=gen).mul_(0.004).half())
    x = torch.randn((1, 4096), device="cuda", generator=gen).half()
    layers = [Case(T, 64, 2048, 1408, 2048, 128, torch.float16, torch.float32, T) for T in (1, 7)]
    bias = torch.zeros(64, device="cuda")  # (with a bias the first kernel hands the ids over)
    fused = lambda: awq.awq_gemm_fused(x, *w, None, 128)  # noqa: E731  (K splits: sums in the scratch)
    kinds = [[lambda c=c, b=b: c.run(8, bias=b) for c in layers for b in (None, bias)], [fused, fused]]
    want = [[f() for f in calls] for calls in kinds]
    torch.cuda.synchronize()
    wrong = [-1, -1]

    def calls(i):
        got = [[f() for f in kinds[i]] for _ in range(200)]
        torch.cuda.synchronize()
        wrong[i] = sum(not torch.equal(y, v) for ys in got for y, v in zip(ys, want[i]))

    threads = [threading.Thread(target=calls, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == [0, 0]


def test_streams_from_outside():
    """A stream that torch did not make: nothing is kept for its handle, the bits are the same."""
    from w4a16_weight_only_amd import scratch

    case = Case(3, 64, 2048, 1408, 2048, 128, torch.bfloat16, torch.bfloat16, 4)
    want = case.run(8)
    torch.cuda.synchronize()
    inner = torch.cuda.Stream()
    outside = torch.cuda.ExternalStream(inner.cuda_stream)
    kept = dict(scratch._kept.blocks)
    kept.pop((0, inner.cuda_stream), None)
    scratch._kept.blocks = dict(kept)
    with torch.cuda.stream(outside):
        got = [case.run(8) for _ in range(20)]
    outside.synchronize()
    assert all(torch.equal(y, want) for y in got) and scratch._kept.blocks.keys() == kept.keys()
    with torch.cuda.stream(inner):
        got = [case.run(8) for _ in range(20)]
    inner.synchronize()
    assert all(torch.equal(y, want) for y in got) and (0, inner.cuda_stream) in scratch._kept.blocks


def test_empty_and_refusals():
    case = Case(9, 8, 256, 96, 288, 32, torch.float16, torch.float16, 1)
    call = lambda x=case.x, router=case.router, up=case.up.dev, down=case.down.dev, topk=2, g=32, **k: awq.awq_moe_layer(  # noqa: E731
        x, router, up, down, topk, g, **k)
    assert call(x=case.x[:0]).shape == (0, 288)
    for error, bad in [
        (ValueError, lambda: call(topk=8)),  # 72 slots
        (ValueError, lambda: call(topk=9)),
        (ValueError, lambda: call(topk=0)),
        (ValueError, lambda: call(groups=3)),
        (ValueError, lambda: call(score="tanh")),
        (ValueError, lambda: call(router=case.router[:, :128].contiguous())),
        (ValueError, lambda: call(router=case.router[:7])),
        (TypeError, lambda: call(router=case.router.bfloat16())),
        (TypeError, lambda: call(x=case.x.float())),
        (ValueError, lambda: call(router=case.router.t().contiguous().t())),
        (ValueError, lambda: call(bias=torch.zeros(7, device="cuda"))),
        (TypeError, lambda: call(bias=torch.zeros(8, device="cuda").half())),
        (ValueError, lambda: call(residual=case.residual[:8])),
        (TypeError, lambda: call(residual=case.residual.float())),
        (ValueError, lambda: call(g=64)),
        (ValueError, lambda: call(down=case.up.dev)),
        (ValueError, lambda: call(down=tuple(t[:7] for t in case.down.dev))),
        (ValueError, lambda: call(out=case.x)),
    ]:
        with pytest.raises(error):
            bad()
    buf = torch.zeros(9 * 288 + 64, dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError):
        call(residual=buf[:9 * 288].view(9, 288), out=buf[64:].view(9, 288))
