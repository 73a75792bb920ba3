"""Dense products with their epilogue: torch tensors in, C ABI calls out.

Work runs on the current stream of the tensors' device.  Where K is split, a call needs scratch
memory, and counters that are zero between calls (scratch.py); calls may be captured into graphs
without a call before.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from .linear import _check_tensor, validate
from .moe import _TYPES, _is, _output
from .scratch import counters_and_scratch

_ACTIVATIONS = {None: _lib.AWQ_ACT_NONE, "relu": _lib.AWQ_ACT_RELU, "silu": _lib.AWQ_ACT_SILU,
                "gelu": _lib.AWQ_ACT_GELU, "gelu_tanh": _lib.AWQ_ACT_GELU_TANH}

_plans = {}  # (workspace, counter) bytes by device and the call's sizes


def _plan(device, *sizes):
    """(workspace, counter) bytes of these sizes on the device, the current one."""
    key = (device.index, sizes)
    need = _plans.get(key)
    if need is None:
        ws, count = ctypes.c_int64(), ctypes.c_int64()
        status = _lib.load().awq_gemm_fused_plan(*sizes, ctypes.byref(ws), ctypes.byref(count))
        _lib.check(status, "awq_gemm_fused_plan")
        if len(_plans) >= 4096:
            _plans.clear()
        _plans[key] = need = (ws.value, count.value)
    return need


def awq_gemm_fused(x: torch.Tensor, qweight: torch.Tensor, qzeros: torch.Tensor, scales: torch.Tensor,
                   bias: torch.Tensor | None = None, group_size: int = 128, *, activation: str | None = None,
                   gated: bool = False, residual: torch.Tensor | None = None, scale: float = 1.0,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """A product with its epilogue, in x's type (fp16 or bfloat16), rounded once:

        y = residual + scale * f(x . dequant(W) + bias)

    f: None (the value itself), "relu", "silu", "gelu" or "gelu_tanh".  gated: the weight (and bias)
    holds the gate's columns, then as many of the up projection's, and f(gate) * up stands in f's
    place.  x may have leading dimensions, as for awq_gemm; residual has y's shape, and out may be
    residual itself."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    dtype, dev = x.dtype, x.device
    if dtype is not torch.float16 and dtype is not torch.bfloat16:
        raise TypeError(f"x must be float16 or bfloat16, got {dtype}")
    if dev.type != "cuda" or not x.is_contiguous():
        _check_tensor("x", x, dtype)
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation must be None, 'relu', 'silu', 'gelu' or 'gelu_tanh', got {activation!r}")
    if not (_is(qweight, torch.int32, dev) and _is(qzeros, torch.int32, dev) and _is(scales, torch.float16, dev)):
        _check_tensor("qweight", qweight, torch.int32, dev)
        _check_tensor("qzeros", qzeros, torch.int32, dev)
        _check_tensor("scales", scales, torch.float16, dev)
    if x.dim() < 1 or qweight.dim() != 2 or qzeros.dim() != 2 or scales.dim() != 2:
        raise ValueError("x must have rows; qweight, qzeros and scales must be 2-D")
    K, words = qweight.shape
    C = 8 * words
    lead = x.shape[:-1]
    if x.shape[-1] != K:
        raise ValueError(f"x has {x.shape[-1]} input features, qweight has {K}")
    G = 1 if group_size == -1 else K // group_size if group_size > 0 else 0
    if K < 1 or qzeros.shape != (G, words) or scales.shape != (G, C):
        validate(K, C, group_size, qweight, qzeros, scales)
    N = C
    if gated:
        if C % 16 != 0:
            raise ValueError("gated: the columns must be two equal halves of whole words")
        N = C // 2
    if bias is not None:
        if not _is(bias, dtype, dev):
            _check_tensor("bias", bias, dtype, dev)
        if bias.shape != (C,):
            raise ValueError(f"bias must be [{C}]")
    shape = lead + (N,)
    if residual is not None:
        if not _is(residual, dtype, dev):
            _check_tensor("residual", residual, dtype, dev)
        if residual.shape != shape:
            raise ValueError(f"residual must be {list(shape)}")
    M = x.numel() // K
    if out is None:
        out = torch.empty_like(residual) if residual is not None else torch.empty(shape, dtype=dtype, device=dev)
    else:
        out = _output(out, shape, dtype, dev)
    sizes = (M, K, N, group_size, 1 if gated else 0)
    if torch.cuda.current_device() == dev.index:
        _launch(x, qweight, qzeros, scales, bias, activation, residual, scale, out, sizes)
    else:
        with torch.cuda.device(dev):
            _launch(x, qweight, qzeros, scales, bias, activation, residual, scale, out, sizes)
    return out


def _launch(x, qweight, qzeros, scales, bias, activation, residual, scale, out, sizes):
    dev = x.device
    M, K, N, group_size, gated = sizes
    ws_bytes, count_bytes = _plan(dev, *sizes)
    counters = ws = hold = None
    if count_bytes:
        counters, ws, hold = counters_and_scratch(dev, count_bytes, ws_bytes)
    elif ws_bytes:
        hold = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
        ws = hold.data_ptr()
    status = _lib.load().awq_gemm_fused(
        x.data_ptr(), _TYPES[x.dtype], qweight.data_ptr(), qzeros.data_ptr(), scales.data_ptr(),
        None if bias is None else bias.data_ptr(), _ACTIVATIONS[activation], gated,
        None if residual is None else residual.data_ptr(), scale, M, K, N, group_size, out.data_ptr(), ws, ws_bytes,
        counters, count_bytes, torch._C._cuda_getCurrentRawStream(dev.index))
    if status != 0:
        _lib.check(status, "awq_gemm_fused")
    del hold
