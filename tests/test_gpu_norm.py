"""awq_norm and awq_add_norm against the formulas in float64.

Tolerances, elementwise, from the arithmetic.  u = 2^-24, q half a step of the output's type, tiny
half its smallest step.  A sum over a row adds at most 32 values a lane, then folds 6 times in a
wave and over up to 16 waves: at most D = 54 roundings of each term.
  statistics  a sum of squares is off by D u of itself, its root's quotient by (D / 2 + 5) u; a mean
              by D u mean|v|, and what is left of v - mean carries that and u (|v| + |mean|).
  n = norm(v) of values off by dv: off by e = inv (dv + dm) + |n| ((D / 2 + 6) u + inv rms(dv + dm)),
              dm = D u mean|v| + mean(dv) + u (|v| + |mean|) with a mean, else 0.  (A change dv of the
              row changes its root mean square by at most rms(dv).)
  z = n w + b: |w| e + 4 u (|n w| + |b|);   r = residual + scale gate z: |scale gate| dz + 4 u (|residual|
              + |scale gate z|), rounded: + q |r| + tiny;   y from n(r) as z: + q |y| + tiny.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import w4a16_weight_only_amd as awq

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}
D = 54
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a HIP GPU")
    awq.load_library()


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def normed(v, dv, weight, bias, kind, unit):
    """norm(v) * weight + bias of v off by dv, and how far that is off."""
    mean = v.mean(axis=1, keepdims=True) if kind == "layer" else 0.0 * v[:, :1]
    dm = D * U * np.abs(v).mean(axis=1, keepdims=True) + dv.mean(axis=1, keepdims=True) + U * (np.abs(v) + np.abs(mean))
    dm = dm if kind == "layer" else 0.0 * v
    inv = 1.0 / np.sqrt(((v - mean) ** 2).mean(axis=1, keepdims=True) + EPS)
    n = (v - mean) * inv
    e = inv * (dv + dm) + np.abs(n) * ((D / 2 + 6) * U + inv * np.sqrt(((dv + dm) ** 2).mean(axis=1, keepdims=True)))
    w = f64(weight) + (1.0 if unit else 0.0)
    b = 0.0 if bias is None else f64(bias)
    return n * w + b, np.abs(w) * e + 4 * U * (np.abs(n * w) + np.abs(b))


def expected(x, residual, weight, bias, gate, scale, pw, pb, kind, unit):
    v = f64(x).reshape(-1, x.shape[-1])
    dv = np.zeros_like(v)
    if pw is not None:
        v, dv = normed(v, dv, pw, pb, kind, unit)
    factor = np.full_like(v, scale)
    if gate is not None:
        rows = f64(gate).reshape(-1, v.shape[1])
        factor = scale * np.repeat(rows, v.shape[0] // rows.shape[0], axis=0)
    res = np.zeros_like(v) if residual is None else f64(residual).reshape(v.shape)
    r = res + factor * v
    dr = np.abs(factor) * dv + 4 * U * (np.abs(res) + np.abs(factor * v))
    if residual is None and gate is None and scale == 1.0:
        dr = dv
    y, dy = normed(r, dr, weight, bias, kind, unit)
    return (r, dr), (y, dy)


def close(got, want, off, where):
    g = f64(got).reshape(want.shape)
    allow = off + HALF[got.dtype] * np.abs(want) + TINY[got.dtype]
    bad = ~(np.abs(g - want) <= allow)
    assert not bad.any(), f"{where}: {bad.sum()} of {bad.size}, worst {np.nanmax(np.abs(g - want) / allow):.3g}"


def make(T, H, dtype, stream, seed, gate=0, bias=False, post=False, unit=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    base = 0.0 if unit else 1.0
    return dict(x=normal(T, H).to(dtype), residual=(2.0 * normal(T, H) + 0.3).to(stream),
                weight=(base + 0.3 * normal(H)).to(dtype), bias=normal(H).to(dtype) if bias else None,
                gate=normal(gate, H).to(dtype) if gate else None,
                pw=(base + 0.3 * normal(H)).to(dtype) if post else None, pb=normal(H).to(dtype) if post and bias else None)


def check(t, kind, scale, unit, where):
    y, r = awq.awq_add_norm(t["x"], t["residual"], t["weight"], t["bias"], gate=t["gate"], scale=scale,
                            post_weight=t["pw"], post_bias=t["pb"], kind=kind, eps=EPS, unit_offset=unit)
    assert y.dtype == t["x"].dtype and r.dtype == t["residual"].dtype and y.shape == r.shape == t["x"].shape
    (rw, dr), (yw, dy) = expected(t["x"], t["residual"], t["weight"], t["bias"], t["gate"], scale, t["pw"], t["pb"],
                                  kind, unit)
    close(r, rw, dr, where + " r")
    close(y, yw, dy, where + " y")


SIZES = [(1, 1), (3, 7), (5, 8), (9, 64), (2, 511), (7, 512), (4, 513), (6, 1000), (5, 1024), (3, 1032), (2, 2047),
         (3, 2048), (2, 4095), (3, 4096), (2, 8192), (3, 8200), (2, 16384), (2, 20001), (2, 32768)]


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,H", SIZES)
def test_sizes(T, H, dtype, kind):
    for i, stream in enumerate((dtype, torch.float32)):
        check(make(T, H, dtype, stream, 100 * H + T + i, gate=(0, T)[i], bias=bool(i), post=not i), kind, (0.5, 1.0)[i],
              bool(i), f"{T}x{H} {dtype} {kind} {stream}")
    t = make(T, H, dtype, dtype, H, bias=True)
    y = awq.awq_norm(t["x"], t["weight"], t["bias"], kind=kind, eps=EPS)
    _, (yw, dy) = expected(t["x"], None, t["weight"], t["bias"], None, 1.0, None, None, kind, False)
    close(y, yw, dy, "norm")


@pytest.mark.parametrize("gate", [0, 1, 2, 6])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("unit", [False, True])
def test_parts(gate, post, bias, unit):
    for kind in ("rms", "layer"):
        check(make(6, 264, torch.bfloat16, torch.bfloat16, gate + 7, gate, bias, post, unit), kind, 1.5, unit, kind)


def test_many_rows():
    check(make(5003, 384, torch.float16, torch.float32, 3, post=True), "rms", 1.0, False, "5003 rows")


def test_more_rows_than_a_launch_holds():
    """2^24 rows of 256 threads each are 2^32 work-items, one too many: the last row is a second launch's."""
    T, H = 1 << 24, 1032
    if torch.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("needs 48 GiB of free device memory")
    gen = torch.Generator(device="cuda").manual_seed(9)
    rows = torch.tensor([0, 1, 12345, 1 << 22, T - 3, T - 2, T - 1], device="cuda")
    some, weight = (torch.randn(s, device="cuda", generator=gen).half() for s in ((len(rows), H), (H,)))
    x = torch.zeros((T, H), dtype=torch.float16, device="cuda")
    x[rows] = some
    y = awq.awq_norm(x, weight, eps=EPS, out=x)
    _, (want, dy) = expected(some, None, weight, None, None, 1.0, None, None, "rms", False)
    close(y[rows], want, dy, "y")
    y[rows] = 0
    for at in range(0, T, 1 << 21):  # rows of zeros stay zeros
        assert not y[at:at + (1 << 21)].view(torch.int64).any()
    del x, y
    torch.cuda.empty_cache()


@pytest.mark.parametrize("H", [96, 1500, 4096])
def test_rows_apart_and_unaligned(H):
    """Rows of a wider tensor, and pointers that are aligned to an element only."""
    for shift, width in ((0, H + 8), (8, H + 24), (1, H + 3)):
        t = make(4, H, torch.float16, torch.float16, H + shift)
        for name in ("x", "residual"):
            wide = torch.randn(4, width, device="cuda").half()
            wide[:, shift:shift + H] = t[name]
            t[name] = wide[:, shift:shift + H]
            assert not t[name].is_contiguous()
        flat = torch.empty(H + 1, dtype=torch.float16, device="cuda")
        flat[1:] = t["weight"]
        t["weight"] = flat[1:]
        check(t, "layer", 1.0, False, f"shift {shift}")


def test_leading_dimensions_and_empty():
    t = make(12, 128, torch.float16, torch.float16, 5)
    y0, r0 = awq.awq_add_norm(t["x"], t["residual"], t["weight"])
    y, r = awq.awq_add_norm(t["x"].view(3, 4, 128), t["residual"].view(3, 4, 128), t["weight"])
    assert y.shape == (3, 4, 128) and torch.equal(y.view(12, 128), y0) and torch.equal(r.view(12, 128), r0)
    empty = torch.empty(0, 128, dtype=torch.float16, device="cuda")
    y, r = awq.awq_add_norm(empty, empty, t["weight"])
    assert y.shape == (0, 128) and r.shape == (0, 128)
    v = awq.awq_norm(t["x"][0], t["weight"])
    assert torch.equal(v, awq.awq_norm(t["x"], t["weight"])[0])


@pytest.mark.parametrize("H", [40, 4096, 9001])
def test_special_values(H):
    """What is not finite stays in its row; a row of zeros is its bias."""
    t = make(6, H, torch.float16, torch.float32, 11, bias=True)
    clean, _ = awq.awq_add_norm(t["x"], t["residual"], t["weight"], t["bias"])
    t["x"][1, H // 2] = float("nan")
    t["residual"][3, H - 1] = float("inf")
    t["x"][4] = 0.0
    t["residual"][4] = 0.0
    y, r = awq.awq_add_norm(t["x"], t["residual"], t["weight"], t["bias"])
    assert torch.isnan(y[1]).all() and torch.isnan(r[1, H // 2]) and torch.isnan(y[3, H - 1])
    assert torch.equal(y[4], t["bias"])
    for row in (0, 2, 5):
        assert torch.equal(y[row], clean[row])


@pytest.mark.parametrize("H", [100, 2048, 5000])
def test_in_place(H):
    t = make(5, H, torch.bfloat16, torch.bfloat16, 2, post=True)
    y, r = awq.awq_add_norm(t["x"], t["residual"], t["weight"], post_weight=t["pw"])
    y2, r2 = awq.awq_add_norm(t["x"], t["residual"], t["weight"], post_weight=t["pw"], out=(t["x"], t["residual"]))
    assert y2 is t["x"] and r2 is t["residual"]
    assert torch.equal(y2, y) and torch.equal(r2, r)


def test_overlaps_are_refused():
    buf = torch.randn(40, 64, device="cuda").half()
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    x, res = buf[:8], buf[8:16]
    for out in ((buf[1:9], buf[24:32]), (buf[16:24], buf[9:17]), (buf[16:24], buf[17:25]), (buf[8:16], buf[24:32]),
                (buf[16:24], buf[:8])):
        with pytest.raises(ValueError):
            awq.awq_add_norm(x, res, w, out=out)
    with pytest.raises(ValueError):
        awq.awq_norm(buf[:8], buf[3], out=buf[:8])


def test_refusals():
    x = torch.zeros(4, 64, dtype=torch.float16, device="cuda")
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    for error, call in [
        (TypeError, lambda: awq.awq_norm(x.float(), w)),
        (TypeError, lambda: awq.awq_norm(x, None)),
        (TypeError, lambda: awq.awq_norm(x, w.bfloat16())),
        (ValueError, lambda: awq.awq_norm(x, w[:32])),
        (ValueError, lambda: awq.awq_norm(x, w, kind="batch")),
        (ValueError, lambda: awq.awq_norm(x.t(), w)),
        (ValueError, lambda: awq.awq_norm(x.cpu(), w)),
        (ValueError, lambda: awq.awq_norm(x[:1].expand(4, 64), w)),
        (TypeError, lambda: awq.awq_add_norm(x, None, w)),
        (TypeError, lambda: awq.awq_add_norm(x, x.bfloat16(), w)),
        (ValueError, lambda: awq.awq_add_norm(x, x[:2], w)),
        (ValueError, lambda: awq.awq_add_norm(x, x, w, post_bias=w)),
        (ValueError, lambda: awq.awq_add_norm(x, x, w, gate=torch.zeros(3, 64, dtype=torch.float16, device="cuda"))),
        (TypeError, lambda: awq.awq_add_norm(x, x, w, gate=torch.zeros(4, 64, device="cuda"))),
        (TypeError, lambda: awq.awq_add_norm(x, x, w, out=(torch.empty_like(x), torch.empty_like(x).float()))),
        (ValueError, lambda: awq.awq_norm(torch.zeros(1, 32776, dtype=torch.float16, device="cuda"),
                                          torch.zeros(32776, dtype=torch.float16, device="cuda"))),
    ]:
        with pytest.raises(error):
            call()


def test_graph_and_streams():
    t = make(7, 4096, torch.float16, torch.float16, 9, gate=7)
    call = lambda: awq.awq_add_norm(t["x"], t["residual"], t["weight"], gate=t["gate"])  # noqa: E731
    y0, r0 = call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, r = call()
    for k in range(3):
        t["x"].mul_(0.5)
        want = call()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(r, want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = call()
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
