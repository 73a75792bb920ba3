"""Two host threads' calls on one stream (the default one): calls that are several launches with the library's
workspace between them give each thread the bits that they give it alone."""
from __future__ import annotations

import threading

import pytest
import torch

import w4a16_weight_only_amd as awq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a HIP GPU")
    awq.load_library()


def packed(K, N, g, seed, *lead):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    words = lambda *shape: torch.randint(-(1 << 31), 1 << 31, lead + shape, dtype=torch.int32, device="cuda", generator=gen)  # noqa: E731
    return words(K, N // 8), words(K // g, N // 8), torch.rand(lead + (K // g, N), device="cuda", generator=gen).mul_(0.01).half()


def rand(*shape, seed):
    return torch.randn(shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))


def side_by_side(kinds, rounds=150):
    """kinds: for each thread its calls; each thread's results against those it gets alone."""
    want = [[f() for f in calls] for calls in kinds]
    torch.cuda.synchronize()
    wrong = [-1] * len(kinds)

    def run(i):
        got = [[f() for f in kinds[i]] for _ in range(rounds)]
        torch.cuda.synchronize()
        same = lambda a, b: all(map(torch.equal, a, b)) if isinstance(a, tuple) else torch.equal(a, b)  # noqa: E731
        wrong[i] = sum(not same(y, v) for ys in got for y, v in zip(ys, want[i]))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(kinds))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == [0] * len(kinds)


def test_splits_joined_by_a_kernel_more():
    """awq_gemm's row tiles with K splits: fp32 sums from the first launch to the second."""
    K, N = 11008, 1024
    w = packed(K, N, 128, 1)
    assert awq.plan(64, K, N, 128)["family"] == "tile" and awq.plan(64, K, N, 128)["splits"] > 1
    assert awq.plan(128, K, N, 128)["family"] == "tile" and awq.plan(128, K, N, 128)["splits"] > 1
    kinds = [[lambda x=rand(M, K, seed=M + s).to(t): awq.awq_gemm(x, *w, None, 128)
              for M in (64, 128) for t in (torch.float16, torch.bfloat16)] for s in (0, 1)]
    side_by_side(kinds)


def test_slots_sorted_by_a_kernel_before():
    """awq_moe_gemm of many tokens: the alignment's table from the first launch to the second."""
    E, K, N = 8, 256, 512
    w = packed(K, N, 64, 2, E)
    gen = torch.Generator(device="cuda").manual_seed(3)
    ids = lambda T: torch.randint(0, E, (T, 2), dtype=torch.int32, device="cuda", generator=gen)  # noqa: E731
    kinds = [[lambda x=rand(T, K, seed=T).half(), i=ids(T): awq.awq_moe_gemm(x, *w, i, 64) for T in sizes]
             for sizes in ((40, 150), (300, 24))]
    side_by_side(kinds)


def test_writer_beside_products():
    """awq_quantize_rtn's scratch is the products' partial sums' buffer."""
    K, N = 11008, 1024
    w, x = packed(K, N, 128, 4), rand(64, K, seed=5).half()
    source = [rand(2048, 512, seed=6).half(), rand(1024, 1024, seed=7).half()]
    side_by_side([[lambda: awq.awq_gemm(x, *w, None, 128)], [lambda s=s: awq.awq_quantize_rtn(s, -1) for s in source]])
