"""awq_gemm_fused and awq_norm where offsets pass 32 bits: tensors of more than 4 GiB, rows further apart than that.
Formulas and tolerances are those of test_gpu_fused.py and test_gpu_norm.py, at chosen rows; the other rows hold
zeros, whose outputs are known."""
from __future__ import annotations

import pytest
import torch

import w4a16_weight_only_amd as awq
from tests import test_gpu_fused as fused
from tests import test_gpu_norm as norm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a HIP GPU")
    awq.load_library()
    yield
    torch.cuda.empty_cache()


def random(*shape, seed, dtype):
    return torch.randn(shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)).to(dtype)


@pytest.mark.parametrize("M,K,N,gated", [(540_001, 4096, 64, False), (540_001, 4096, 32, True), (1_100_003, 32, 2080, False)],
                         ids=["x", "x-gated", "y"])
def test_products(M, K, N, gated):
    """x, or y and the residual, of more than 4 GiB."""
    dtype = torch.bfloat16
    C = 2 * N if gated else N
    w, b = fused.Weight(K, C, 32, 1), random(C, seed=2, dtype=dtype)
    rows = torch.tensor([0, 1, 255, 256, M // 2, M - 300, M - 2, M - 1], device="cuda")
    x, r = torch.zeros((M, K), dtype=dtype, device="cuda"), torch.zeros((M, N), dtype=dtype, device="cuda")
    x[rows], r[rows] = random(len(rows), K, seed=3, dtype=dtype), random(len(rows), N, seed=4, dtype=dtype)
    y = awq.awq_gemm_fused(x, *w.dev, b, 32, activation="silu", gated=gated, residual=r, out=r)
    want = fused.expected(x[rows], w, b, "silu", gated, None, 1.0)
    residual = random(len(rows), N, seed=4, dtype=dtype).double()
    off = want[1] + 3 * fused.U * (residual.abs() + want[0].abs())
    fused.close(y[rows], want[0] + residual, off, "rows")
    rest = awq.awq_gemm_fused(x[2:3].contiguous(), *w.dev, b, 32, activation="silu", gated=gated)  # a row of zeros
    y[rows] = rest
    step = 1 << 18
    for at in range(0, M, step):  # f(b) alone, rounded once: off by no more than a step from the other kernel's
        part = y[at:at + step]
        same = part == rest
        assert bool((same | ((part.float() - rest.float()).abs() <= 2 * fused.HALF[dtype] * rest.float().abs())).all())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_norm_of_rows_far_apart(dtype):
    H, apart = 1032, (1 << 31) + 8
    flat = torch.empty(2 * apart + H, dtype=dtype, device="cuda")
    x = flat.as_strided((3, H), (apart, 1))
    x.copy_(random(3, H, seed=5, dtype=dtype))
    weight, residual = random(H, seed=6, dtype=dtype), random(3, H, seed=7, dtype=torch.float32)
    y, r = awq.awq_add_norm(x, residual, weight, kind="layer", eps=norm.EPS)
    (want_r, dr), (want, dy) = norm.expected(x.contiguous(), residual, weight, None, None, 1.0, None, None, "layer", False)
    norm.close(r, want_r, dr, "r")
    norm.close(y, want, dy, "y")
