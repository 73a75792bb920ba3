"""awq_moe_gate_up, awq_moe_down, awq_moe_mlp and AwqMoe against the oracle in float64.

Tolerances, elementwise, from the arithmetic.  u = 2^-24 (half a step of fp32), r half a step
of the activation type (2^-11 fp16, 2^-8 bfloat16), tiny its smallest step's half.
  A product of K terms is a sum of exact terms in fp32, its running value multiplied by a
  quotient of scales at each of the G group boundaries (three roundings, one of them a
  reciprocal good to two of u): at most (K + 4 G + 4) roundings of something no larger than
  A = sum |x| |W|, so it is off by dP = (K + 4 G + 4) u A.
  For bfloat16 A is sum |x| (143 + 143) s, that of sums corrected for the zeros afterwards
  (x . (128 + q) - (128 + z) x . 1): wider than products of q - z need, which these now are.
  h = silu(g) u: |silu'| <= 1.1, so dh = 1.1 dP_g |u| + |silu(g)| dP_u + dP_g dP_u + 8 u |h|
  (exp, quotient, product), then r |h| + tiny for the rounding.
  y = sum_j w_j v_j: sum |w_j| dP_j + (topk + 2) u sum |w_j| |v_j| + r |y| + tiny.
awq_moe_mlp must give awq_moe_down of awq_moe_gate_up bit for bit: it runs the same products.  With
at most 8 slots, or up to 64 and fewer than 12 per expert, it keeps h as two terms instead, rounded and what that
left out (itself rounded: r r |h| + tiny): dh without the rounding, plus that, through |W|, and 2 K
terms in the second product.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import w4a16_weight_only_amd as awq
from oracle import awq_ref as oracle
from w4a16_weight_only_amd import synth

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a HIP GPU")
    awq.load_library()


class Layer:
    """Packed weights of E experts, K -> N, on the device and as float64 matrices."""

    def __init__(self, E, K, N, g, seed, edit=None):
        rng = np.random.default_rng(seed)
        G = 1 if g == -1 else K // g
        self.g = g
        self.G = G
        self.qw = synth.random_words(rng, (E, K, N // 8))
        self.qz = synth.random_words(rng, (E, G, N // 8))
        self.sc = (rng.uniform(0.5, 1.5, (E, G, N)) / (6.5 * np.sqrt(K))).astype(np.float16)
        if edit is not None:
            edit(self)
        self.dev = tuple(torch.from_numpy(a).cuda() for a in (self.qw, self.qz, self.sc))
        self.W = np.stack([oracle.dequant_ref(self.qw[e], self.qz[e], self.sc[e], g) for e in range(E)]).astype(np.float64)
        # |W| as the corrected form meets it: (143 + 143) s.
        self.C = np.repeat(286.0 * np.abs(self.sc.astype(np.float64)), K // G, axis=1)


def f64(t):
    return t.double().cpu().numpy()


def activations(shape, dtype, seed):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape)).to(dtype).cuda()


def routing(T, E, topk, seed):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(E)[:topk] if topk <= E else rng.integers(0, E, topk) for _ in range(T)])
    w = rng.uniform(0.1, 1.0, (T, topk)).astype(np.float32)
    return torch.from_numpy(ids.astype(np.int32)).cuda(), torch.from_numpy(w).cuda()


def product(rows, layer, ids, dtype):
    """rows [S, K] by experts ids [S]: the values, and how far fp32 may leave them."""
    S, K = rows.shape
    E, N = layer.W.shape[0], layer.W.shape[2]
    v, d = np.zeros((S, N)), np.zeros((S, N))
    A = np.abs(layer.W) if dtype == torch.float16 else layer.C
    for e in range(E):
        m = ids == e
        if m.any():
            v[m] = rows[m] @ layer.W[e]
            d[m] = (K + 4 * layer.G + 4) * U * (np.abs(rows[m]) @ A[e])
    return v, d


def gate_up_ref(x, layer, ids, dtype):
    topk = ids.shape[1]
    v, d = product(np.repeat(f64(x), topk, axis=0), layer, f64(ids).ravel(), dtype)
    (g, u), (dg, du) = np.split(v, 2, axis=1), np.split(d, 2, axis=1)
    s = g / (1 + np.exp(-g))
    h = s * u
    dh = 1.1 * dg * np.abs(u) + np.abs(s) * du + dg * du + 8 * U * np.abs(h)
    return h, dh + HALF[dtype] * (np.abs(h) + dh) + TINY[dtype]


def down_ref(h, layer, ids, weights, dtype):
    T, topk = ids.shape
    flat = f64(ids).ravel()
    v, d = product(f64(h), layer, flat, dtype)
    live = (flat >= 0) & (flat < layer.W.shape[0])
    w = np.where(live, f64(weights).ravel(), 0.0)[:, None]
    fold = lambda a: a.reshape(T, topk, -1).sum(axis=1)  # noqa: E731
    y = fold(w * v)
    dy = fold(np.abs(w) * d) + (topk + 2) * U * fold(np.abs(w * v))
    return y, dy + HALF[dtype] * (np.abs(y) + dy) + TINY[dtype]


def two_terms(ids, layer):
    S, E = ids.numel(), layer.W.shape[0]
    return S <= 8 or S <= 64 and S < 12 * E


def mlp_ref(x, up, down, ids, weights, dtype):
    """The whole MLP where h has two terms."""
    h, tol = gate_up_ref(x, up, ids, dtype)
    r = HALF[dtype]
    dh = (tol - TINY[dtype] - r * np.abs(h)) / (1 + r)  # without the rounding
    dh = dh + r * r * (np.abs(h) + dh) + TINY[dtype]
    T, topk = ids.shape
    flat = f64(ids).ravel()
    w = np.where((flat >= 0) & (flat < down.W.shape[0]), f64(weights).ravel(), 0.0)[:, None]
    v, d = product(h, down, flat, dtype)
    A = np.abs(down.W)
    for e in range(A.shape[0]):
        m = flat == e
        if m.any():
            d[m] = 2 * d[m] * (1 + 2 * r) + dh[m] @ A[e]
    fold = lambda a: a.reshape(T, topk, -1).sum(axis=1)  # noqa: E731
    y = fold(w * v)
    dy = fold(np.abs(w) * d) + (topk + 2) * U * fold(np.abs(w * v))
    return y, dy + r * (np.abs(y) + dy) + TINY[dtype]


def check_mlp(x, up, down, ids, weights, g, steps, dtype):
    """awq_moe_mlp against its two steps' bits, or the two-term definition."""
    y = awq.awq_moe_mlp(x, up.dev, down.dev, ids, weights, g)
    if two_terms(ids, up):
        close(y, *mlp_ref(x, up, down, ids, weights, dtype), "mlp")
    else:
        assert torch.equal(y, steps)
    return y


def close(got, ref, tol, label):
    err = np.abs(f64(got) - ref)
    worst = float((err / tol).max()) if err.size else 0.0
    print(f"[{label}] max err {err.max() if err.size else 0:.3e}, {worst:.3f} of the tolerance", flush=True)
    assert np.isfinite(f64(got)).all(), label
    assert (err <= tol).all(), (label, worst)


# (T, E, topk, K, inner, N, g)
CASES = [
    (1, 1, 1, 32, 32, 32, 32),            # the smallest layer, K below one k-tile
    (1, 8, 2, 512, 192, 256, 128),        # one token
    (2, 4, 2, 96, 64, 96, 32),            # K % 64 = 32
    (1, 16, 4, 1024, 352, 544, 64),
    (3, 5, 3, 320, 160, 288, 160),        # a group that ends inside a k-tile
    (4, 8, 2, 768, 416, 96, -1),
    (5, 64, 8, 256, 128, 160, 128),       # most experts idle
    (7, 3, 2, 288, 96, 64, 96),
    (16, 8, 2, 1024, 256, 512, 128),
    (17, 8, 2, 256, 224, 320, 32),
    (31, 60, 4, 256, 96, 128, 64),
    (48, 4, 4, 512, 128, 256, 64),        # every token to every expert
    (64, 16, 4, 256, 160, 192, -1),
    (129, 2, 1, 352, 288, 416, 32),
    (130, 1, 1, 256, 128, 256, 128),      # one expert: a dense gated MLP
    (200, 8, 2, 512, 384, 352, 128),
    (300, 4, 2, 128, 64, 64, 64),
    (513, 8, 3, 192, 96, 224, 64),
]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("T,E,topk,K,inner,N,g", CASES)
def test_against_the_oracle(T, E, topk, K, inner, N, g, dtype):
    print(f"experts T={T} E={E} topk={topk} K={K} inner={inner} N={N} g={g} {dtype}", flush=True)
    g2 = g if g != -1 and inner % g == 0 else -1
    if g2 != g:
        up, down = Layer(E, K, 2 * inner, g, 1), Layer(E, inner, N, g2, 2)
    else:
        up, down = Layer(E, K, 2 * inner, g, 1), Layer(E, inner, N, g, 2)
    x = activations((T, K), dtype, T + K)
    ids, w = routing(T, E, topk, T + E)
    h = awq.awq_moe_gate_up(x, *up.dev, ids, g)
    close(h, *gate_up_ref(x, up, ids, dtype), "gate_up")
    y = awq.awq_moe_down(h, *down.dev, ids, w, g2)
    close(y, *down_ref(h, down, ids, w, dtype), "down")
    if g2 == g:
        check_mlp(x, up, down, ids, w, g, y, dtype)


def big(T, E, topk, K, inner, N, g, dtype, seed):
    up, down = Layer(E, K, 2 * inner, g, seed), Layer(E, inner, N, g, seed + 1)
    ids, w = routing(T, E, topk, seed)
    return up, down, activations((T, K), dtype, seed), ids, w


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("T,E,topk,K,inner,N,g", [(1, 4, 2, 4096, 1024, 512, 128), (9, 4, 2, 2048, 2816, 1024, 64),
                                                  (70, 6, 2, 4096, 512, 2048, 128), (1, 2, 1, 11008, 64, 64, 64)])
def test_long_axes(T, E, topk, K, inner, N, g, dtype):
    up, down, x, ids, w = big(T, E, topk, K, inner, N, g, dtype, 21)
    h = awq.awq_moe_gate_up(x, *up.dev, ids, g)
    close(h, *gate_up_ref(x, up, ids, dtype), "gate_up")
    y = awq.awq_moe_down(h, *down.dev, ids, w, g)
    close(y, *down_ref(h, down, ids, w, dtype), "down")
    check_mlp(x, up, down, ids, w, g, y, dtype)


# Row tiles: more than 72 slots per expert, and enough columns that the tiles fill a third of the
# card.  Rows per expert around every height of a tile (64, 128, 192, 256), one more than one,
# none, a few.
COUNTS = [(300, 190, 0, 130, 100, 64, 20, 1), (512, 257, 193, 129, 65), (256, 192, 128, 64)]


def routed_by_counts(counts, seed):
    """topk 1: counts[e] tokens of expert e, shuffled."""
    ids = np.random.default_rng(seed).permutation(np.repeat(np.arange(len(counts)), counts)).astype(np.int32)
    w = np.random.default_rng(seed + 1).uniform(0.1, 1.0, (ids.size, 1)).astype(np.float32)
    return torch.from_numpy(ids[:, None]).cuda(), torch.from_numpy(w).cuda()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("counts", COUNTS, ids=["eight", "five", "four"])
@pytest.mark.parametrize("K,g", [(32, 32), (96, 32), (160, 160), (320, 64), (256, 128), (288, 96), (384, 128), (480, -1)])
def test_row_tiles(K, g, counts, dtype):
    E, T = len(counts), sum(counts)
    print(f"row tiles K={K} g={g} counts={counts} {dtype}", flush=True)
    ids, w = routed_by_counts(counts, K)
    x = activations((T, K), dtype, K + 1)
    up = Layer(E, K, 2 * 4512, g, 3)
    close(awq.awq_moe_gate_up(x, *up.dev, ids, g), *gate_up_ref(x, up, ids, dtype), "gate_up")
    down = Layer(E, K, 8736, g, 4)
    close(awq.awq_moe_down(x, *down.dev, ids, w, g), *down_ref(x, down, ids, w, dtype), "down")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
def test_row_tiles_odd_scales_and_slots(dtype):
    """Zero and negative scales, unrouted slots and a token's repeated expert on row tiles."""
    T, E, topk, K, g, N = 420, 4, 2, 160, 32, 9120
    up, down = Layer(E, K, 2 * 4544, g, 5, odd_scales), Layer(E, K, N, g, 6, odd_scales)
    ids, w = routing(T, E, topk, 7)
    ids[3], ids[5, 1], ids[9] = torch.tensor([-1, E]), E + 3, torch.tensor([2, 2])
    w[3] = float("nan")
    x, h = activations((T, K), dtype, 8), activations((T * topk, K), dtype, 9)
    live = ((ids >= 0) & (ids < E)).flatten()
    out = torch.full((T * topk, 4544), 7.0, dtype=dtype, device="cuda")
    awq.awq_moe_gate_up(x, *up.dev, ids, g, out=out)
    assert (out[~live] == 7.0).all() and torch.equal(out[18], out[19])
    ref, tol = gate_up_ref(x, up, ids, dtype)
    m = live.cpu().numpy()
    close(out[live], ref[m], tol[m], "gate_up")
    y = awq.awq_moe_down(h, *down.dev, ids, w, g)
    assert (y[3] == 0).all()
    close(y, *down_ref(h, down, ids, w, dtype), "down")


@pytest.mark.parametrize("T,E,topk,K,inner,N", [(9000, 4, 2, 64, 32, 64), (700, 3, 25, 32, 32, 32)])
def test_more_slots_than_the_alignment_holds(T, E, topk, K, inner, N):
    """Over 16384 slots: the alignment counts those beyond in a second pass."""
    up, down = Layer(E, K, 2 * inner, 32, 8), Layer(E, inner, N, 32, 9)
    x = activations((T, K), torch.float16, 10)
    ids, w = routing(T, E, topk, 11)
    h = awq.awq_moe_gate_up(x, *up.dev, ids, 32)
    close(h, *gate_up_ref(x, up, ids, torch.float16), "gate_up")
    close(awq.awq_moe_down(h, *down.dev, ids, w, 32), *down_ref(h, down, ids, w, torch.float16), "down")


@pytest.mark.parametrize("seed", range(12))
def test_drawn(seed):
    """Sizes, types, routing and group sizes drawn at random."""
    rng = np.random.default_rng(500 + seed)
    g = int(rng.choice([32, 64, 96, 128, -1]))
    step = 32 if g == -1 else g
    E = int(rng.choice([1, 2, 7, 16, 33]))
    topk = int(rng.integers(1, min(E, 6) + 1))
    T = int(np.exp(rng.uniform(0, np.log(400))))
    K, inner = step * int(rng.integers(1, max(2, 640 // step))), step * int(rng.integers(1, max(2, 512 // step)))
    N = 32 * int(rng.integers(1, 24))
    dtype = torch.float16 if seed % 2 else torch.bfloat16
    print(f"drawn T={T} E={E} topk={topk} K={K} inner={inner} N={N} g={g} {dtype}", flush=True)
    up, down, x, ids, w = big(T, E, topk, K, inner, N, g, dtype, seed)
    h = awq.awq_moe_gate_up(x, *up.dev, ids, g)
    close(h, *gate_up_ref(x, up, ids, dtype), "gate_up")
    y = awq.awq_moe_down(h, *down.dev, ids, w, g)
    close(y, *down_ref(h, down, ids, w, dtype), "down")
    check_mlp(x, up, down, ids, w, g, y, dtype)


def odd_scales(layer):
    """Scales of zero (single groups, both signs, whole columns), negative ones, and neighbours
    at both ends of fp16's range within one column."""
    s, G = layer.sc, layer.sc.shape[1]
    s[:, 0, ::7] = 0.0
    s[:, 3 % G, 1::5] = -0.0
    s[:, -1, 2::9] = 0.0
    s[1, :, 4::11] = 0.0
    s[:, 2 % G] *= -1
    s[:, 4 % G, 6::13] = 6e-8
    s[:, 1 % G, 6::13] = 0.01
    s[:, 2 % G, 6::13] = 6e-8


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("T", [2, 40, 300])
def test_odd_scales(T, dtype):
    K, inner, N, g, E = 256, 64, 96, 32, 3
    up, down = Layer(E, K, 2 * inner, g, 31, odd_scales), Layer(E, K, N, g, 32, odd_scales)
    x, h = activations((T, K), dtype, 5), activations((T * 2, K), dtype, 6)
    ids, w = routing(T, E, 2, 7)
    close(awq.awq_moe_gate_up(x, *up.dev, ids, g), *gate_up_ref(x, up, ids, dtype), "gate_up")
    close(awq.awq_moe_down(h, *down.dev, ids, w, g), *down_ref(h, down, ids, w, dtype), "down")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("T", [1, 9, 16])
def test_h_of_two_terms(T, dtype):
    """Few slots: y is off by its own rounding and hardly more, also with half of the slots' ids not
    routed."""
    E, topk, K, inner, N, g = 128, 4, 512, 512, 768, 64
    up, down, x, ids, w = big(T, E, topk, K, inner, N, g, dtype, 131)
    for some in (False, True):
        if some:
            ids[:, 2:] = -1
        y = awq.awq_moe_mlp(x, up.dev, down.dev, ids, w, g)
        ref, tol = mlp_ref(x, up, down, ids, w, dtype)
        close(y, ref, tol, "mlp")
        once = torch.from_numpy(ref).to(dtype).double().numpy() - ref
        ratio = np.linalg.norm(f64(y) - ref) / np.linalg.norm(once)
        print(f"error {ratio:.3f} of one rounding", flush=True)
        assert ratio < 1.1


def test_h_of_two_terms_past_the_types_range():
    """An h that rounds to infinity, or is none: its second term is nothing, not minus infinity."""
    E, K, inner, N, g = 2, 64, 32, 64, 32
    up, down, x, ids, w = big(2, E, 1, K, inner, N, g, torch.float16, 141)
    ids.fill_(1)
    x[0] *= 1000.0
    h = awq.awq_moe_gate_up(x, *up.dev, ids, g)
    assert torch.isinf(h[0]).any() and torch.isfinite(h[1]).all()
    steps = awq.awq_moe_down(h, *down.dev, ids, w, g)
    y = awq.awq_moe_mlp(x, up.dev, down.dev, ids, w, g)
    assert torch.equal(torch.isnan(y[0]), torch.isnan(steps[0])) and torch.isfinite(y[1]).all()
    x[0, 3] = float("nan")
    assert torch.isnan(awq.awq_moe_mlp(x, up.dev, down.dev, ids, w, g)[0]).all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("T", [1, 3, 40, 150])
def test_unrouted_and_repeated_slots(T, dtype):
    """Ids outside [0, E): h rows stay as they were, y gets nothing from them (zeros where a
    token has no other), whatever their weight.  One expert twice in a token counts twice."""
    E, topk, K, inner, N, g = 4, 3, 256, 96, 64, 64
    up, down = Layer(E, K, 2 * inner, g, 41), Layer(E, inner, N, 32, 42)
    x = activations((T, K), dtype, 8)
    ids, w = routing(T, E, topk, 9)
    ids[0] = torch.tensor([-1, E, 1 << 30])
    w[0] = float("nan")
    if T > 1:
        ids[1] = torch.tensor([2, 2, -7])
        w[1, 2] = float("inf")
        ids[T - 1, 0] = E
    h = torch.full((T * topk, inner), 7.0, dtype=dtype, device="cuda")
    awq.awq_moe_gate_up(x, *up.dev, ids, g, out=h)
    live = ((ids >= 0) & (ids < E)).flatten()
    assert (h[~live] == 7.0).all()
    ref, tol = gate_up_ref(x, up, ids, dtype)
    m = live.cpu().numpy()
    close(h[live], ref[m], tol[m], "gate_up")
    if T > 1:
        assert torch.equal(h[topk], h[topk + 1])
    y = torch.full((T + 1, N), 3.0, dtype=dtype, device="cuda")  # a row behind the last token
    awq.awq_moe_down(h, *down.dev, ids, w, 32, out=y[:T])
    assert (y[0] == 0).all() and (y[T] == 3.0).all()
    close(y[:T], *down_ref(h, down, ids, w, dtype), "down")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("T,E,topk", [(1, 4, 3), (7, 2, 5), (40, 4, 3), (64, 1, 1)])
def test_mlp_of_unrouted_and_repeated_slots(T, E, topk, dtype):
    """The whole MLP: zeros for a token without a routed slot, whatever its weights hold and the
    workspace held; more slots per token than experts; every slot unrouted."""
    K, inner, N, g = 64, 96, 64, 32
    up, down = Layer(E, K, 2 * inner, g, 43), Layer(E, inner, N, g, 44)
    x = activations((T, K), dtype, 45)
    ids, w = routing(T, E, topk, 46)
    ids[T - 1] = E
    w[T - 1] = float("nan")
    junk = torch.full((1 << 22,), float("nan"), device="cuda")  # what the allocator hands out next
    del junk
    steps = awq.awq_moe_down(awq.awq_moe_gate_up(x, *up.dev, ids, g), *down.dev, ids, w, g)
    y = check_mlp(x, up, down, ids, w, g, steps, dtype)
    assert (y[T - 1] == 0).all()
    ids.fill_(-1)
    assert (awq.awq_moe_mlp(x, up.dev, down.dev, ids, w, g) == 0).all()


@pytest.mark.parametrize("T", [2, 20, 200])
def test_all_slots_on_one_expert(T):
    E, K, inner, N, g = 6, 512, 160, 96, 32
    up, down, x, ids, w = big(T, E, 2, K, inner, N, g, torch.float16, 51)
    ids.fill_(4)
    h = awq.awq_moe_gate_up(x, *up.dev, ids, g)
    close(h, *gate_up_ref(x, up, ids, torch.float16), "gate_up")
    close(awq.awq_moe_down(h, *down.dev, ids, w, g), *down_ref(h, down, ids, w, torch.float16), "down")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("T", [3, 40, 150])
def test_nonfinite_rows_stay_apart(T, dtype):
    """NaN and infinities in one token's x (or h): its outputs are not finite somewhere, every
    other token's bits are those of the clean call; so too rows of x that are not routed."""
    E, topk, K, inner, N, g = 4, 2, 288, 96, 64, 96
    up, down = Layer(E, K, 2 * inner, g, 61), Layer(E, inner, N, g, 62)
    x = activations((T, K), dtype, 11)
    ids, w = routing(T, E, topk, 12)
    ids[2] = -1
    clean_h = awq.awq_moe_gate_up(x, *up.dev, ids, g)
    clean_y = awq.awq_moe_mlp(x, up.dev, down.dev, ids, w, g)
    for bad, at in ((float("nan"), 0), (float("inf"), K - 1), (-float("inf"), 255)):
        y = x.clone()
        y[1, at] = bad
        y[2] = bad
        h = awq.awq_moe_gate_up(y, *up.dev, ids, g)
        m = awq.awq_moe_mlp(y, up.dev, down.dev, ids, w, g)
        rows = torch.ones(T * topk, dtype=torch.bool)
        rows[2:6] = False  # token 1's rows, and token 2's, which are not written
        assert torch.equal(h[rows], clean_h[rows])
        assert not torch.isfinite(h[2:4]).all()
        keep = torch.arange(T) != 1
        assert torch.equal(m[keep], clean_y[keep])
        assert not torch.isfinite(m[1]).all()


def test_empty_batch():
    up, down = Layer(2, 64, 64, 32, 71), Layer(2, 32, 32, 32, 72)
    x = torch.zeros(0, 64, dtype=torch.float16, device="cuda")
    ids, w = torch.zeros(0, 2, dtype=torch.int32, device="cuda"), torch.zeros(0, 2, device="cuda")
    assert awq.awq_moe_gate_up(x, *up.dev, ids, 32).shape == (0, 32)
    assert awq.awq_moe_down(x[:, :32].contiguous(), *down.dev, ids, w, 32).shape == (0, 32)
    assert awq.awq_moe_mlp(x, up.dev, down.dev, ids, w, 32).shape == (0, 32)


@pytest.mark.parametrize("T", [1, 12, 90, 260])
def test_graph_replays_side_by_side(T):
    """Two graphs captured on one stream, with no eager call before, replayed on two streams at
    once: each has its own workspace.  Every replay gives the eager bits, on new inputs too."""
    E, topk, K, inner, N, g = 8, 2, 512, 256, 384, 128
    up, down, x, ids, w = big(T, E, topk, K, inner, N, g, torch.float16, 81)
    xs = [x, activations((T, K), torch.float16, 82)]
    ys = [torch.empty(T, N, dtype=torch.float16, device="cuda") for _ in xs]
    graphs = []
    for v, y in zip(xs, ys):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            awq.awq_moe_mlp(v, up.dev, down.dev, ids, w, g, out=y)
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(4):
        for v in xs:
            v.mul_(0.75)
        want = [awq.awq_moe_mlp(v, up.dev, down.dev, ids, w, g) for v in xs]
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ys, want))


@pytest.mark.parametrize("T", [1, 12, 90])
def test_two_streams_at_once(T):
    up, down, x, ids, w = big(T, 8, 2, 512, 256, 384, 128, torch.bfloat16, 91)
    want = awq.awq_moe_mlp(x, up.dev, down.dev, ids, w, 128)
    torch.cuda.synchronize()
    got = []
    for s in [torch.cuda.Stream() for _ in range(3)]:
        with torch.cuda.stream(s):
            got += [awq.awq_moe_mlp(x, up.dev, down.dev, ids, w, 128) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(v, want) for v in got)


def test_row_tiles_in_graphs_and_on_streams():
    """Row tiles: graphs replayed side by side on two streams while a third works eagerly, each
    replay the eager bits."""
    T, E, topk, K, inner, N, g = 400, 2, 2, 64, 4352, 8704, 64
    gen = torch.Generator(device="cuda").manual_seed(95)

    def packed(rows, cols):
        words = lambda *shape: torch.randint(-2 ** 31, 2 ** 31, shape, generator=gen, device="cuda").int()  # noqa: E731
        sc = (torch.rand(E, rows // g, cols, generator=gen, device="cuda") + 0.5) / (6.5 * rows ** 0.5)
        return words(E, rows, cols // 8), words(E, rows // g, cols // 8), sc.half()

    up, down = packed(K, 2 * inner), packed(inner, N)
    ids, w = routing(T, E, topk, 96)
    xs = [activations((T, K), torch.bfloat16, 97 + i) for i in range(2)]
    ys = [torch.empty(T, N, dtype=torch.bfloat16, device="cuda") for _ in xs]
    graphs = []
    for x, y in zip(xs, ys):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            awq.awq_moe_mlp(x, up, down, ids, w, g, out=y)
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(4):
        for x in xs:
            x.mul_(0.75)
        want = [awq.awq_moe_mlp(x, up, down, ids, w, g) for x in xs]
        assert all(v.float().std() > 0 for v in want)
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        with torch.cuda.stream(streams[2]):
            eager = awq.awq_moe_mlp(xs[1], up, down, ids, w, g)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ys + [eager], want + want[1:]))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("T", [1, 33])
def test_layer_module(T, dtype):
    """Router, routing and MLP together: the module, its steps one by one, and the oracle."""
    E, topk, K, inner, g = 16, 4, 256, 128, 64
    up, down = Layer(E, K, 2 * inner, g, 101), Layer(E, inner, K, g, 102)
    router = activations((E, K), dtype, 103) / 16
    bias = torch.linspace(-0.1, 0.1, E).cuda()
    layer = awq.AwqMoe(router, up.dev, down.dev, topk, g, bias=bias, score="sigmoid", groups=4, topk_groups=2,
                       group_top=2, scale=2.0)
    x = activations((T, 1, K), dtype, 104)
    y = layer(x)
    assert y.shape == (T, 1, K) and y.dtype == dtype
    logits = torch.nn.functional.linear(x[:, 0], router)
    w, ids = awq.awq_moe_route(logits, topk, score="sigmoid", bias=bias, groups=4, topk_groups=2, group_top=2, scale=2.0)
    wr, ir = oracle.route_ref(f64(logits), topk, score="sigmoid", bias=f64(bias), groups=4, topk_groups=2, group_top=2,
                              scale=2.0)
    assert np.array_equal(ids.cpu().numpy(), ir)
    h = awq.awq_moe_gate_up(x[:, 0].contiguous(), *up.dev, ids, g)
    steps = awq.awq_moe_down(h, *down.dev, ids, w, g)
    assert torch.equal(y[:, 0], check_mlp(x[:, 0].contiguous(), up, down, ids, w, g, steps, dtype))
    close(steps, *down_ref(h, down, ids, w, dtype), "layer")


def test_refusals():
    up, down, x, ids, w = big(4, 3, 2, 128, 64, 96, 32, torch.float16, 111)
    qw, qz, sc = up.dev
    bad = [
        lambda: awq.awq_moe_gate_up(x[:, :64], *up.dev, ids, 32),                # not contiguous, wrong K
        lambda: awq.awq_moe_gate_up(x[:3], *up.dev, ids, 32),                    # ids of another T
        lambda: awq.awq_moe_gate_up(x, *up.dev, ids.flatten(), 32),
        lambda: awq.awq_moe_gate_up(x, qw[0], qz[0], sc[0], ids, 32),            # one expert, not stacked
        lambda: awq.awq_moe_gate_up(x, qw, qz[:2], sc, ids, 32),
        lambda: awq.awq_moe_gate_up(x, *up.dev, ids, 64),                        # zeros of another group size
        lambda: awq.awq_moe_gate_up(x, *up.dev, ids, 32, out=torch.empty(8, 65, dtype=torch.float16, device="cuda")),
        lambda: awq.awq_moe_gate_up(x.t(), *up.dev, ids, 32),
        lambda: awq.awq_moe_down(x, *up.dev, ids, w, 32),                        # 4 rows for 8 slots
        lambda: awq.awq_moe_down(x[:4], *up.dev, ids[:2], w, 32),                # weights of another T
        lambda: awq.awq_moe_mlp(x, up.dev, up.dev, ids, w, 32),                  # down's K is not inner
        lambda: awq.awq_moe_mlp(x, up.dev, tuple(t[:2] for t in down.dev), ids, w, 32),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: awq.awq_moe_gate_up(x.float(), *up.dev, ids, 32),
                 lambda: awq.awq_moe_gate_up(x, *up.dev, ids.long(), 32),
                 lambda: awq.awq_moe_mlp(x, up.dev, down.dev, ids, w.half(), 32),
                 lambda: awq.awq_moe_mlp(x, up.dev, down.dev, ids, w, 32,
                                         out=torch.empty(4, 96, dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(TypeError):
            call()
