"""A decoder block's dense feed-forward half on AWQ GEMM-layout weights."""
from __future__ import annotations

import torch

from .fused import awq_gemm_fused
from .norm import awq_add_norm, awq_norm


class AwqMlp(torch.nn.Module):
    """Inference-only feed-forward block on the residual stream:

        y = x + scale * post(down(f(up(norm(x)))))

    up and down are packed weights (qweight, qzeros, scales).  With gated the first holds the gate's
    columns, then the up projection's, and f(gate) * up stands in f's place; activation is
    awq_gemm_fused's.  norm and post_norm are weights of norms before and after, or None; kind, eps
    and unit_offset are awq_norm's.

    forward(x, normed=None, then=None): normed is norm(x), where the block before has formed it; then
    is the weight of the norm that follows (of the same kind): (that norm of y, y) comes back, the
    residual, post_norm and the norm in one pass.  Without then and post_norm the residual is
    joined by the second product."""

    def __init__(self, up, down, group_size=128, *, activation="silu", gated=True, up_bias=None, down_bias=None,
                 norm=None, post_norm=None, kind="rms", eps=1e-6, unit_offset=False, scale=1.0):
        super().__init__()
        for name, layer in (("up", up), ("down", down)):
            for part, t in zip(("qweight", "qzeros", "scales"), layer):
                self.register_buffer(f"{name}_{part}", t)
        self.register_buffer("up_bias", up_bias)
        self.register_buffer("down_bias", down_bias)
        self.register_buffer("norm", norm)
        self.register_buffer("post_norm", post_norm)
        self.group_size = group_size
        self.activation = activation
        self.gated = gated
        self.norms = dict(kind=kind, eps=eps, unit_offset=unit_offset)
        self.scale = scale

    def forward(self, x, normed=None, then=None):
        if normed is not None and (self.norm is None or normed.shape != x.shape or normed.dtype is not x.dtype):
            raise ValueError("normed must be norm(x), of x's shape and type, of a block with a norm")
        x = x.contiguous()
        h = x if self.norm is None else awq_norm(x, self.norm, **self.norms) if normed is None else normed.contiguous()
        h = awq_gemm_fused(h, self.up_qweight, self.up_qzeros, self.up_scales, self.up_bias, self.group_size,
                           activation=self.activation, gated=self.gated)
        down = (self.down_qweight, self.down_qzeros, self.down_scales, self.down_bias, self.group_size)
        if self.post_norm is None and then is None:
            return awq_gemm_fused(h, *down, residual=x, scale=self.scale)
        z = awq_gemm_fused(h, *down)
        normed, y = awq_add_norm(z, x, then, scale=self.scale, post_weight=self.post_norm, **self.norms)
        return y if then is None else (normed, y)
