"""The modules' handling of what they hold, on the CPU."""
from __future__ import annotations

import io

import pytest
import torch

import w4a16_weight_only_amd as awq


def packed(K, N, *lead):
    return (torch.zeros(lead + (K, N // 8), dtype=torch.int32), torch.zeros(lead + (1, N // 8), dtype=torch.int32),
            torch.ones(lead + (1, N), dtype=torch.float16))


def saved_and_loaded(module, *without):
    """A module saved whole by a version that had no such attributes."""
    for name in without:
        del module.__dict__[name]
    f = io.BytesIO()
    torch.save(module, f)
    f.seek(0)
    return torch.load(f, weights_only=False)


def test_modules_saved_before_their_options(monkeypatch):
    """Their calls are those of a module without the options."""
    calls = []
    monkeypatch.setattr("w4a16_weight_only_amd.linear.awq_gemm", lambda x, *rest: calls.append("gemm") or x)
    linear = saved_and_loaded(awq.AwqLinear(*packed(32, 32), group_size=-1), "activation")
    x = torch.ones(3, 32, dtype=torch.float16)
    assert torch.equal(linear(x), x) and calls == ["gemm"]
    monkeypatch.setattr("w4a16_weight_only_amd.moe.awq_moe_route", lambda *a, **k: calls.append("route") or (None, None))
    monkeypatch.setattr("w4a16_weight_only_amd.moe.awq_moe_mlp", lambda x, *a, **k: calls.append("mlp") or x)
    layer = saved_and_loaded(awq.AwqMoe(torch.ones(4, 32, dtype=torch.float16), packed(32, 64, 4), packed(32, 32, 4), 2,
                                        -1), "one_call")
    assert torch.equal(layer(x), x) and calls == ["gemm", "route", "mlp"]


def test_a_norm_that_the_block_does_not_have_is_refused():
    """AwqMlp.forward's normed stands for norm(x); without a norm it would be left out."""
    mlp = awq.AwqMlp(packed(32, 64), packed(32, 32), -1)
    x = torch.ones(3, 32, dtype=torch.float16)
    with pytest.raises(ValueError, match="normed"):
        mlp(x, normed=x)
    for wrong in (x[:2], x.float()):
        with pytest.raises(ValueError, match="normed"):
            awq.AwqMlp(packed(32, 64), packed(32, 32), -1, norm=torch.ones(32, dtype=torch.float16))(x, normed=wrong)
