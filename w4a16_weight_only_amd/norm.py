"""Norms on the residual stream, before and after a block: torch tensors in, C ABI calls out."""
from __future__ import annotations

import torch

from . import _lib
from .linear import _check_tensor
from .moe import _TYPES, _call, _is, _output

_KINDS = {"rms": _lib.AWQ_RMS, "layer": _lib.AWQ_LAYER}


def _rows(name, t, dtypes, device=None):
    """(rows, elements between them) of a tensor whose rows are its last dimension: contiguous, or
    2-D with adjacent elements."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype in dtypes and t.is_cuda and t.is_contiguous() and (device is None or t.device == device):
        shape = t.shape
        if len(shape) == 2 and shape[1] >= 1:
            return shape
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a HIP device, got {t.device}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dim() < 1 or t.shape[-1] < 1:
        raise ValueError(f"{name} must have rows of at least one element")
    H = t.shape[-1]
    if t.is_contiguous():
        return t.numel() // H, H
    if t.dim() != 2 or (H > 1 and t.stride(1) != 1) or (t.shape[0] > 1 and t.stride(0) < H):
        raise ValueError(f"{name} must be contiguous, or 2-D with adjacent elements in a row")
    return t.shape[0], t.stride(0) if t.shape[0] > 1 else H


def _vector(name, t, H, dtype, device):
    if t is None:
        return None
    if not _is(t, dtype, device):
        _check_tensor(name, t, dtype, device)
    if t.shape != (H,):
        raise ValueError(f"{name} must be [{H}]")
    return t.data_ptr()


def _run(x, residual, weight, bias, gate, scale, post_weight, post_bias, kind, eps, unit_offset, y, r, keep_r):
    T, x_stride = _rows("x", x, (torch.float16, torch.bfloat16))
    H, dtype, dev = x.shape[-1], x.dtype, x.device
    if kind not in _KINDS:
        raise ValueError(f"kind must be 'rms' or 'layer', got {kind!r}")
    if weight is None and (bias is not None or not keep_r or y is not None):
        raise TypeError("weight must be a torch.Tensor")
    if post_bias is not None and post_weight is None:
        raise ValueError("post_bias needs post_weight")
    stream_type, residual_stride = dtype, H
    if residual is not None:
        rows, residual_stride = _rows("residual", residual, (dtype, torch.float32), dev)
        if residual.shape != x.shape:
            raise ValueError(f"residual must be {list(x.shape)}, got {list(residual.shape)}")
        stream_type = residual.dtype
    gates = 0
    if gate is not None:
        if not _is(gate, dtype, dev):
            _check_tensor("gate", gate, dtype, dev)
        gates = gate.numel() // H
        if gate.dim() not in (1, 2) or gate.shape[-1] != H or gates < 1 or T % gates != 0:
            raise ValueError(f"gate must be [{H}], or [B, {H}] with B a divisor of the {T} rows")
    vectors = [_vector(n, t, H, dtype, dev) for n, t in (("post_weight", post_weight), ("post_bias", post_bias),
                                                         ("weight", weight), ("bias", bias))]
    whole = x_stride == H  # then x is contiguous
    if weight is not None:
        y = torch.empty_like(x) if y is None and whole else _output(y, x.shape, dtype, dev)
    if keep_r:
        whole = residual_stride == H
        r = torch.empty_like(residual) if r is None and whole else _output(r, x.shape, stream_type, dev)
    _call(_lib.load().awq_add_norm, "awq_add_norm", dev, x.data_ptr(), _TYPES[dtype], T, H, x_stride,
          None if residual is None else residual.data_ptr(), _TYPES[stream_type], residual_stride,
          None if gate is None else gate.data_ptr(), gates, scale, *vectors, _KINDS[kind], 1 if unit_offset else 0, eps,
          None if y is None else y.data_ptr(), r.data_ptr() if keep_r else None)
    return y, r


def awq_norm(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, *, kind: str = "rms",
             eps: float = 1e-6, unit_offset: bool = False, out: torch.Tensor | None = None) -> torch.Tensor:
    """y = norm(x) * weight + bias over the last dimension, in x's type (fp16 or bfloat16): kind
    "rms", v / sqrt(mean(v^2) + eps), or "layer", the same of v - mean(v).  unit_offset: 1 + weight
    in weight's place.  x is contiguous, or 2-D with rows apart; out may be x itself."""
    return _run(x, None, weight, bias, None, 1.0, None, None, kind, eps, unit_offset, out, None, False)[0]


def awq_add_norm(x: torch.Tensor, residual: torch.Tensor, weight: torch.Tensor | None, bias: torch.Tensor | None = None, *,
                 gate: torch.Tensor | None = None, scale: float = 1.0, post_weight: torch.Tensor | None = None,
                 post_bias: torch.Tensor | None = None, kind: str = "rms", eps: float = 1e-6,
                 unit_offset: bool = False, out: tuple | None = None) -> tuple:
    """Between two blocks: x, the first one's output (fp16 or bfloat16), joins the residual stream (of
    x's type or fp32), which is normed for the second: (y, r),

        r = residual + scale * gate * z,  z = x or, with post_weight, norm(x) * post_weight + post_bias
        y = norm(r) * weight + bias       (of r before it is rounded to residual's type)

    With weight None there is no second norm, and y is None.  kind, eps and unit_offset as for
    awq_norm, for both norms.  gate: [H], or [B, H] for B equal runs
    of rows (sequences, or with B = T every row).  out, if given, is (y, r) to write into: r may be
    residual itself, y may be x itself."""
    if residual is None:
        raise TypeError("residual must be a torch.Tensor")
    y, r = out if out is not None else (None, None)
    return _run(x, residual, weight, bias, gate, scale, post_weight, post_bias, kind, eps, unit_offset, y, r, True)
