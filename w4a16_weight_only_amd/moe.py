"""Routed-expert layers on AWQ GEMM-layout weights: routing, the gated MLP and its halves.

Like linear.py this module marshals torch tensors into the C ABI and computes nothing
itself.  A packed weight is the triple (qweight, qzeros, scales) stacked over the experts:
int32 [E, K, N/8], int32 [E, G, N/8], fp16 [E, G, N].  Work runs on the current stream of
the tensors' device; each call's workspace comes from torch's allocator on that stream, so
calls may be captured into graphs without a call before.
"""
from __future__ import annotations

import torch

from . import _lib
from .linear import _check_tensor, validate

_TYPES = {torch.float16: _lib.AWQ_F16, torch.bfloat16: _lib.AWQ_BF16, torch.float32: _lib.AWQ_F32}
_SCORES = {"softmax": _lib.AWQ_SOFTMAX, "sigmoid": _lib.AWQ_SIGMOID}

# A decoding step's calls are a few microseconds each on the GPU, so the checks below look at
# each tensor once and leave the wording of a refusal to functions that only a refusal reaches.


def _is(t, dtype, device):
    """A contiguous tensor of this type on this device."""
    return isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == device and t.is_contiguous()


def _check_act(name, t):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.float16 and t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be float16 or bfloat16, got {t.dtype}")
    if t.device.type != "cuda" or not t.is_contiguous():
        _check_tensor(name, t, t.dtype)
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")


def _check_layer(name, layer, K, group_size, device):
    """The packed weight's experts and columns."""
    qweight, qzeros, scales = layer
    if _is(qweight, torch.int32, device) and _is(qzeros, torch.int32, device) and _is(scales, torch.float16, device):
        shape = qweight.shape
        if len(shape) == 3 and shape[1] == K and K > 0:
            E, _, words = shape
            G = 1 if group_size == -1 else K // group_size if group_size > 0 else 0
            if qzeros.shape == (E, G, words) and scales.shape == (E, G, 8 * words):
                return E, 8 * words  # a group size that does not divide K is the library's to refuse
    _refuse_layer(name, qweight, qzeros, scales, K, group_size, device)


def _refuse_layer(name, qweight, qzeros, scales, K, group_size, device):
    _check_tensor(f"{name} qweight", qweight, torch.int32, device)
    _check_tensor(f"{name} qzeros", qzeros, torch.int32, device)
    _check_tensor(f"{name} scales", scales, torch.float16, device)
    if qweight.dim() != 3 or qzeros.dim() != 3 or scales.dim() != 3:
        raise ValueError(f"{name}: qweight, qzeros and scales must be stacked per expert")
    E, rows, words = qweight.shape
    if rows != K or qzeros.shape[0] != E or scales.shape[0] != E or E < 1:
        raise ValueError(f"{name}: expert weight shapes disagree with each other or with {K} input features")
    validate(K, words * 8, group_size, qweight[0], qzeros[0], scales[0])
    raise ValueError(f"{name}: unsupported shapes")


def _check_ids(expert_ids, device, tokens=None):
    if not _is(expert_ids, torch.int32, device):
        _check_tensor("expert_ids", expert_ids, torch.int32, device)
    shape = expert_ids.shape
    if len(shape) != 2 or (tokens is not None and shape[0] != tokens) or shape[1] < 1:
        raise ValueError("expert_ids must be [T, topk]" + ("" if tokens is None else f" with T = {tokens}"))
    return shape


def _check_weights(weights, ids_shape, device):
    if not _is(weights, torch.float32, device):
        _check_tensor("weights", weights, torch.float32, device)
    if weights.shape != ids_shape:
        raise ValueError(f"weights must be {list(ids_shape)}")


def _output(out, shape, dtype, device):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not _is(out, dtype, device):
        _check_tensor("out", out, dtype, device)
    if out.shape != shape:
        raise ValueError(f"out must be {list(shape)}")
    return out


def _act(t, nan_weights):
    return _TYPES[t.dtype] | (_lib.AWQ_NAN_WEIGHTS if nan_weights else 0)


def _call(fn, name, device, *args):
    """fn(*args, stream) with the tensors' device current; the stream is that device's current one."""
    index = device.index
    if torch.cuda.current_device() == index:
        status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if status != 0:
        _lib.check(status, name)


_sizes = {}  # workspace bytes by device and the call's sizes


def _workspace(device, *sizes):
    """(tensor, bytes) on the current stream.  The size follows from the call's sizes and the
    device's compute units; decoding repeats them, so it is asked for once."""
    key = (device.index, sizes)
    need = _sizes.get(key)
    if need is None:
        with torch.cuda.device(device):
            need = _lib.load().awq_moe_workspace(*sizes)
        if need < 0:
            _lib.check(need, "awq_moe_workspace")
        if len(_sizes) >= 4096:
            _sizes.clear()
        _sizes[key] = need = max(need, 16)
    return torch.empty(need, dtype=torch.uint8, device=device), need


def awq_moe_route(logits: torch.Tensor, topk: int, *, score: str = "softmax", bias: torch.Tensor | None = None,
                  groups: int = 1, topk_groups: int = 1, group_top: int = 1, renormalize: bool = True,
                  scale: float = 1.0, out: tuple | None = None) -> tuple:
    """Each token's topk experts and their weights from router logits [T, E] (fp16, bfloat16
    or fp32; rows may be strided): (weights fp32 [T, topk], expert_ids int32 [T, topk]).

    score "softmax" or "sigmoid"; bias (fp32 [E]) is added to the scores for the choice only;
    of `groups` groups of consecutive experts the best topk_groups are considered, each worth
    its largest score (group_top 1) or the sum of its two largest (group_top 2).  renormalize
    divides the weights by their sum, scale multiplies them.  Ties go to the lowest index.
    An expert with a logit of -inf is never chosen; a slot without an expert gets id -1 and
    weight 0; a row with a NaN gets ids -1 and NaN weights."""
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a torch.Tensor")
    if logits.dtype not in _TYPES:
        raise TypeError(f"logits must be float16, bfloat16 or float32, got {logits.dtype}")
    dev = logits.device
    if dev.type != "cuda":
        raise ValueError(f"logits must be on a HIP device, got {dev}")
    if logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be [T, E] with adjacent experts")
    if score not in _SCORES:
        raise ValueError(f"score must be 'softmax' or 'sigmoid', got {score!r}")
    T, E = logits.shape
    stride = logits.stride(0) if T > 1 else E
    if bias is not None:
        if not _is(bias, torch.float32, dev):
            _check_tensor("bias", bias, torch.float32, dev)
        if bias.shape != (E,):
            raise ValueError(f"bias must be [{E}]")
    if topk < 1:
        raise ValueError("topk must be at least 1")
    weights, ids = out if out is not None else (None, None)
    weights = _output(weights, (T, topk), torch.float32, dev)
    ids = _output(ids, (T, topk), torch.int32, dev)
    _call(_lib.load().awq_moe_route, "awq_moe_route", dev, logits.data_ptr(), _TYPES[logits.dtype], T, E, stride,
          None if bias is None else bias.data_ptr(), _SCORES[score], groups, topk_groups, group_top, topk,
          1 if renormalize else 0, scale, weights.data_ptr(), ids.data_ptr())
    return weights, ids


def awq_moe_gate_up(x: torch.Tensor, qweight: torch.Tensor, qzeros: torch.Tensor, scales: torch.Tensor,
                    expert_ids: torch.Tensor, group_size: int = 128, out: torch.Tensor | None = None) -> torch.Tensor:
    """First half of the gated MLP: x [T, K] (fp16 or bfloat16), weights of 2 I columns (the
    gate's first), expert_ids int32 [T, topk] -> h [T * topk, I] in x's type,
    h[t topk + j] = silu(x[t] . gate) * (x[t] . up) of expert expert_ids[t, j].  Rows of ids
    outside [0, E) keep what `out` holds, which may not overlap x."""
    _check_act("x", x)
    dev = x.device
    T, K = x.shape
    E, N = _check_layer("gate_up", (qweight, qzeros, scales), K, group_size, dev)
    _, topk = _check_ids(expert_ids, dev, T)
    if N % 16 != 0:
        raise ValueError("gate_up: the columns must be two equal halves of whole words")
    inner = N // 2
    out = _output(out, (T * topk, inner), x.dtype, dev)
    ws, nbytes = _workspace(dev, T, topk, E, K, inner, 0, group_size)
    _call(_lib.load().awq_moe_gate_up, "awq_moe_gate_up", dev, x.data_ptr(), _TYPES[x.dtype], qweight.data_ptr(),
          qzeros.data_ptr(), scales.data_ptr(), expert_ids.data_ptr(), T, topk, E, K, inner, group_size,
          out.data_ptr(), ws.data_ptr(), nbytes)
    return out


def awq_moe_down(h: torch.Tensor, qweight: torch.Tensor, qzeros: torch.Tensor, scales: torch.Tensor,
                 expert_ids: torch.Tensor, weights: torch.Tensor, group_size: int = 128,
                 out: torch.Tensor | None = None, nan_weights: bool = False) -> torch.Tensor:
    """Second half: h [T * topk, K], expert_ids int32 and weights fp32 [T, topk] ->
    y [T, N] = sum over j of weights[t, j] * (h[t topk + j] . W[expert_ids[t, j]]) in h's
    type.  Ids outside [0, E) add nothing, whatever their weight; with nan_weights a NaN weight
    makes its token NaN there too, as awq_moe_route leaves a row that has no scores."""
    _check_act("h", h)
    dev = h.device
    S, K = h.shape
    E, N = _check_layer("down", (qweight, qzeros, scales), K, group_size, dev)
    T, topk = _check_ids(expert_ids, dev)
    if T * topk != S:
        raise ValueError(f"expert_ids must name an expert for each of the {S} rows of h")
    _check_weights(weights, expert_ids.shape, dev)
    out = _output(out, (T, N), h.dtype, dev)
    ws, nbytes = _workspace(dev, T, topk, E, 0, K, N, group_size)
    _call(_lib.load().awq_moe_down, "awq_moe_down", dev, h.data_ptr(), _act(h, nan_weights), qweight.data_ptr(),
          qzeros.data_ptr(), scales.data_ptr(), expert_ids.data_ptr(), weights.data_ptr(), T, topk, E, K, N,
          group_size, out.data_ptr(), ws.data_ptr(), nbytes)
    return out


def awq_moe_mlp(x: torch.Tensor, gate_up: tuple, down: tuple, expert_ids: torch.Tensor, weights: torch.Tensor,
                group_size: int = 128, out: torch.Tensor | None = None, nan_weights: bool = False) -> torch.Tensor:
    """The gated MLP of routed experts in one call: x [T, K], gate_up and down packed weights
    (qweight, qzeros, scales) of K -> 2 I and I -> N columns, expert_ids int32 and weights fp32
    [T, topk] -> y [T, N] in x's type.  The same values as awq_moe_down of awq_moe_gate_up, but
    for a decoding step's few slots (up to 64, of which at most 8 or fewer than 12 per expert),
    where h is not rounded on the way (a larger batch in parts of so many slots has that too).  An h
    beyond the type's range is infinite, as awq_moe_gate_up's is.  nan_weights as for awq_moe_down."""
    _check_act("x", x)
    dev = x.device
    T, K = x.shape
    E, wide = _check_layer("gate_up", gate_up, K, group_size, dev)
    if wide % 16 != 0:
        raise ValueError("gate_up: the columns must be two equal halves of whole words")
    inner = wide // 2
    E2, N = _check_layer("down", down, inner, group_size, dev)
    if E2 != E:
        raise ValueError(f"gate_up has {E} experts, down {E2}")
    _, topk = _check_ids(expert_ids, dev, T)
    _check_weights(weights, expert_ids.shape, dev)
    out = _output(out, (T, N), x.dtype, dev)
    ws, nbytes = _workspace(dev, T, topk, E, K, inner, N, group_size)
    _call(_lib.load().awq_moe_mlp, "awq_moe_mlp", dev, x.data_ptr(), _act(x, nan_weights),
          *[t.data_ptr() for t in gate_up], *[t.data_ptr() for t in down], expert_ids.data_ptr(), weights.data_ptr(),
          T, topk, E, K, inner, N, group_size, out.data_ptr(), ws.data_ptr(), nbytes)
    return out


class AwqMoe(torch.nn.Module):
    """Inference-only routed-expert layer: a dense router [E, K] and the experts' packed gate_up and
    down weights.  A router in the activations' type gives logits rounded to it; one in fp32 gives
    fp32 logits, which do not tie experts that are a 16-bit rounding apart.  Routing arguments are awq_moe_route's.  A token
    whose logits hold a NaN (for the softmax, or +inf) comes out as NaN."""

    def __init__(self, router, gate_up, down, topk, group_size=128, bias=None, **routing):
        super().__init__()
        self.register_buffer("router", router)
        self.register_buffer("bias", bias)
        for name, layer in (("gate_up", gate_up), ("down", down)):
            for part, t in zip(("qweight", "qzeros", "scales"), layer):
                self.register_buffer(f"{name}_{part}", t)
        self.topk = topk
        self.group_size = group_size
        self.routing = routing

    def forward(self, x):
        rows = x.reshape(-1, x.shape[-1]).contiguous()
        if self.router.dtype is not rows.dtype and self.router.dtype is not torch.float32:
            raise TypeError(f"router must be {rows.dtype} or float32, got {self.router.dtype}")
        logits = torch.nn.functional.linear(rows.to(self.router.dtype), self.router)
        weights, ids = awq_moe_route(logits, self.topk, bias=self.bias, **self.routing)
        y = awq_moe_mlp(rows, (self.gate_up_qweight, self.gate_up_qzeros, self.gate_up_scales),
                        (self.down_qweight, self.down_qzeros, self.down_scales), ids, weights, self.group_size,
                        nan_weights=True)
        return y.reshape(x.shape[:-1] + (y.shape[-1],))
