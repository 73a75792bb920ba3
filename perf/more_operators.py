"""The measured cases of the operators around the packed products: their inputs, their plain form
in elementary torch operations, and their definition in 64 bits.

  fused  x [M, K] -> y = residual + scale * f(x . W + bias), f an activation; gated (W of 2 I
         columns): f(x . Wg + bg) * (x . Wu + bu) in place of f
  norm   x [T, H] -> r = residual + scale * gate * z, z = x or a norm of x (post), and
         y = norm(r) * weight + bias; norms divide by the root mean square or also take the mean off
  layer  x [T, K] -> y [T, K] = residual + sum over the topk experts, chosen by x . router^T, of
         weight * down(silu(gate(x)) * up(x)), for a few tokens

`own` false: the plain form. `own` true: the framework's entry points.
"""
import math

import numpy as np
import torch

own = False

# Column j of a packed word sits in nibble INVERSE[j].
INVERSE = (0, 4, 1, 5, 2, 6, 3, 7)
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def _fused(name, M, K, N, g, dtype, act="none", gated=False, bias=False, residual=False, scale=1.0):
    """N: columns of y (the weight has twice as many if gated)."""
    return dict(name=name, op="fused", M=M, K=K, N=N, g=g, dtype=dtype, act=act, gated=gated, bias=bias,
                residual=residual, scale=scale)


def _norm(name, T, H, dtype, kind, stream, bias=False, post=False, gate=0, scale=1.0, unit_offset=False):
    """stream: the type of residual and r; gate: its rows (0: none)."""
    return dict(name=name, op="norm", T=T, H=H, dtype=dtype, kind=kind, stream=stream, bias=bias, post=post, gate=gate,
                scale=scale, unit_offset=unit_offset)


def _layer(name, T, E, topk, K, inner, g, dtype, router, score="softmax", bias=False, groups=1, topk_groups=1,
           group_top=1, residual=True, scale=1.0):
    return dict(name=name, op="layer", T=T, E=E, topk=topk, K=K, inner=inner, g=g, dtype=dtype, router=router,
                score=score, bias=bias, groups=groups, topk_groups=topk_groups, group_top=group_top, residual=residual,
                scale=scale)


def listed():
    return [
        # A decoding token's output projection, added to the residual stream.
        _fused("fused_token", 1, 4096, 4096, 128, "f16", bias=True, residual=True),
        # The gate and up projections of an odd decoding batch.
        _fused("fused_gated_batch", 19, 4096, 11008, 128, "bf16", act="silu", gated=True),
        # A short prompt through the first product of a plain two-layer MLP.
        _fused("fused_gelu", 200, 2048, 8192, 64, "f16", act="gelu_tanh", bias=True),
        # A prompt's second product, back into the residual stream, one quantization group.
        _fused("fused_down_prompt", 1000, 11008, 4096, -1, "bf16", residual=True),
        # A prompt's gate and up projections.
        _fused("fused_gated_prompt", 2048, 4096, 11008, 128, "f16", act="silu", gated=True),
        # The norm between two blocks for one decoding token: latency alone.
        _norm("norm_token", 1, 4096, "f16", "rms", "f16"),
        # An odd decoding batch with norms on both sides of the block, weights off one.
        _norm("norm_sandwich", 45, 2048, "bf16", "rms", "bf16", post=True, unit_offset=True),
        # A prompt of eight sequences, each with its gate, on a residual stream of 32 bits.
        _norm("norm_prompt", 8192, 4096, "bf16", "layer", "f32", bias=True, gate=8),
        # A decoding token through a whole layer of 64 experts.
        _layer("layer_token", 1, 64, 8, 2048, 1408, 128, "f16", "f32"),
        # A small batch through it: sigmoid scores, a balancing bias, groups, scaled weights.
        _layer("layer_batch", 7, 64, 8, 2048, 1408, 64, "bf16", "bf16", score="sigmoid", bias=True, groups=8,
               topk_groups=4, group_top=2, scale=2.5),
        # A decoding token, and a batch, through the 8-expert layer.
        _layer("layer_wide_token", 1, 8, 2, 4096, 14336, 128, "bf16", "bf16"),
        _layer("layer_wide_batch", 16, 8, 2, 4096, 14336, 128, "f16", "f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("fused", "norm", "layer"))
    dtype = rng.choice(("f16", "bf16"))
    if op == "norm":
        H = _log(rng, 64, 16384)
        T = _log(rng, 1, max(2, min(16384, 8192 * 4096 // H)))
        rows = rng.choice((0, 0, 1, T, T))
        return _drop_name(_norm("", T, H, dtype, rng.choice(("rms", "layer")), rng.choice((dtype, dtype, "f32")),
                                bias=rng.random() < 0.4, post=rng.random() < 0.4, gate=rows,
                                scale=rng.choice((1.0, 1.0, 0.125)), unit_offset=rng.random() < 0.3))
    g = rng.choice((32, 64, 128, 128, -1))
    step = 32 if g == -1 else g
    size = lambda lo, hi: max(step, _log(rng, lo, hi) // step * step)  # noqa: E731
    if op == "fused":
        K, N = size(256, 11008), _log(rng, 256, 14336) // 32 * 32
        gated = rng.random() < 0.4
        most = 300_000_000_000 // (2 * K * N * (2 if gated else 1))
        return _drop_name(_fused("", _log(rng, 1, max(1, min(4096, most))), K, N, g, dtype,
                                 act=rng.choice(("none", "relu", "silu", "gelu", "gelu_tanh")), gated=gated,
                                 bias=rng.random() < 0.5, residual=rng.random() < 0.5, scale=rng.choice((1.0, 0.5))))
    groups = rng.choice((1, 1, 4))
    E, topk = rng.choice(((8, 2), (16, 4), (60, 4), (64, 8), (128, 8), (32, 1)))
    topk_groups = rng.randint(2, 4) if groups > 1 else 1
    return _drop_name(_layer("", _log(rng, 1, 64 // topk), E, topk, size(512, 4096), size(256, 4096), g, dtype,
                             rng.choice((dtype, "f32")), score=rng.choice(("softmax", "sigmoid")),
                             bias=rng.random() < 0.4, groups=groups, topk_groups=topk_groups,
                             group_top=rng.choice((1, 2)), residual=rng.random() < 0.5, scale=rng.choice((1.0, 2.5))))


def _drop_name(case):
    del case["name"]
    return case


SIZE = {"f16": 2, "bf16": 2, "f32": 4}


def _packed_bytes(K, N, g):
    return K * N // 2 + (1 if g == -1 else K // g) * (N // 2 + 2 * N)


def work(case):
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        vectors = 1 + case["bias"] + case["post"] * (1 + case["bias"]) + case["gate"]
        return {"bytes": T * H * (4 + 2 * SIZE[case["stream"]]) + 2 * H * vectors,
                "flops": T * H * (16 if case["post"] else 10)}
    K, g = case["K"], case["g"]
    if case["op"] == "fused":
        M, N = case["M"], case["N"]
        wide = N * (2 if case["gated"] else 1)
        return {"bytes": _packed_bytes(K, wide, g) + 2 * M * K + 2 * M * N * (1 + case["residual"]) + 2 * wide * case["bias"],
                "flops": 2 * M * K * wide}
    T, E, topk, inner = case["T"], case["E"], case["topk"], case["inner"]
    active = E * (1.0 - (1.0 - topk / E) ** T)  # experts that are read, for even routing
    weights = active * (_packed_bytes(K, 2 * inner, g) + _packed_bytes(inner, K, g))
    return {"bytes": int(weights) + E * K * SIZE[case["router"]] + 2 * T * K * (2 + case["residual"]),
            "flops": 2 * T * E * K + 6 * T * topk * K * inner}


# ---- Inputs.

def _packed(gen, K, N, g, *lead):
    """A packed weight (stacked over `lead`): uniform codes and zeros, scales that keep a product's
    size near its input's (codes less zeros have a spread of about 6.5)."""
    G = 1 if g == -1 else K // g
    words = lambda *shape: torch.randint(-(1 << 31), 1 << 31, lead + shape, dtype=torch.int32, device="cuda", generator=gen)  # noqa: E731
    scales = torch.rand(lead + (G, N), device="cuda", generator=gen).add_(0.5).mul_(1.0 / (6.5 * math.sqrt(K)))
    return words(K, N // 8), words(G, N // 8), scales.half()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, device="cuda", generator=gen)  # noqa: E731
    dtype = TYPES[case["dtype"]]
    state = dict(case=case)
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        # A residual stream larger than what is added to it, with a few channels that stand out.
        stand_out = 1.0 + 20.0 * (torch.rand(H, device="cuda", generator=gen) < 0.01)
        state["x"] = normal(T, H).to(dtype)
        state["residual"] = (3.0 * normal(T, H) * stand_out + 0.2).to(TYPES[case["stream"]])
        around = 0.0 if case["unit_offset"] else 1.0
        state["weight"] = (around + 0.2 * normal(H)).to(dtype)
        state["bias"] = (0.2 * normal(H)).to(dtype) if case["bias"] else None
        state["post_weight"] = (around + 0.2 * normal(H)).to(dtype) if case["post"] else None
        state["post_bias"] = (0.2 * normal(H)).to(dtype) if case["post"] and case["bias"] else None
        state["gate"] = (0.5 + 0.3 * normal(case["gate"], H)).to(dtype) if case["gate"] else None
        return state
    K, g = case["K"], case["g"]
    if case["op"] == "fused":
        M, N = case["M"], case["N"]
        wide = N * (2 if case["gated"] else 1)
        state["x"] = normal(M, K).to(dtype)
        state["weight"] = _packed(gen, K, wide, g)
        state["bias"] = (0.3 * normal(wide)).to(dtype) if case["bias"] else None
        state["residual"] = normal(M, N).to(dtype) if case["residual"] else None
        return state
    T, E, inner = case["T"], case["E"], case["inner"]
    state["x"] = normal(T, K).to(dtype)
    state["router"] = (normal(E, K) * (1.5 / math.sqrt(K))).to(TYPES[case["router"]])
    state["bias"] = 0.2 * normal(E) if case["bias"] else None
    state["gate_up"] = _packed(gen, K, 2 * inner, g, E)
    state["down"] = _packed(gen, inner, K, g, E)
    state["residual"] = normal(T, K).to(dtype) if case["residual"] else None
    return state


# ---- The plain form.

def _dequant(qweight, qzeros, scales):
    """[B, K, N] in 32 bits: (code - zero) * scale."""
    shift = 4 * torch.tensor(INVERSE, dtype=torch.int32, device=qweight.device)
    B, K, words = qweight.shape
    G = qzeros.shape[1]
    q = ((qweight.unsqueeze(-1) >> shift) & 15).view(B, G, K // G, words * 8)
    z = ((qzeros.unsqueeze(-1) >> shift) & 15).view(B, G, 1, words * 8)
    return ((q - z).float() * scales.float().unsqueeze(2)).view(B, K, words * 8)


def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _activation(kind, v):
    if kind == "relu":
        return v.clamp_min(0.0)
    if kind == "silu":
        return _silu(v)
    if kind == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if kind == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _plain_fused(state):
    case, x = state["case"], state["x"]
    v = torch.matmul(x.float(), _dequant(*(t.unsqueeze(0) for t in state["weight"]))[0])
    if state["bias"] is not None:
        v = v + state["bias"].float()
    if case["gated"]:
        v = _activation(case["act"], v[:, :case["N"]]) * v[:, case["N"]:]
    else:
        v = _activation(case["act"], v)
    v = v * case["scale"]
    if state["residual"] is not None:
        v = v + state["residual"].float()
    return v.to(x.dtype)


EPS = 1e-6


def _plain_normed(case, v, weight, bias):
    if case["kind"] == "layer":
        v = v - v.mean(dim=1, keepdim=True)
    v = v / torch.sqrt((v * v).mean(dim=1, keepdim=True) + EPS)
    v = v * (weight.float() + (1.0 if case["unit_offset"] else 0.0))
    return v if bias is None else v + bias.float()


def _plain_norm(state):
    case, x = state["case"], state["x"]
    z = x.float()
    if case["post"]:
        z = _plain_normed(case, z, state["post_weight"], state["post_bias"])
    if state["gate"] is not None:
        z = z * state["gate"].float().repeat_interleave(case["T"] // case["gate"], dim=0)
    r = state["residual"].float() + case["scale"] * z
    return _plain_normed(case, r, state["weight"], state["bias"]).to(x.dtype), r.to(state["residual"].dtype)


def _plain_route(case, logits, bias):
    """(weights, ids) of each token, from logits in 64 bits."""
    T, E = logits.shape
    if case["score"] == "softmax":
        p = torch.exp(logits - logits.amax(dim=1, keepdim=True))
        score = p / p.sum(dim=1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-logits))
    choice = score if bias is None else score + bias.double()
    G = case["groups"]
    if G > 1:
        best = choice.view(T, G, E // G).sort(dim=2, descending=True).values
        worth = best[:, :, 0] + best[:, :, 1] if case["group_top"] == 2 else best[:, :, 0]
        rank = worth.sort(dim=1, descending=True, stable=True).indices
        keep = torch.zeros((T, G), dtype=torch.bool, device=logits.device)
        keep.scatter_(1, rank[:, :case["topk_groups"]], True)
        choice = choice.masked_fill(~keep.repeat_interleave(E // G, dim=1), -math.inf)
    ids = choice.sort(dim=1, descending=True, stable=True).indices[:, :case["topk"]]
    w = score.gather(1, ids)
    return (w / w.sum(dim=1, keepdim=True) * case["scale"]).float(), ids


def _plain_product(rows, layer, ids):
    """rows [T, topk, K] (32 bits), each by its expert ids [T, topk] -> [T, topk, N] (32 bits)."""
    T, topk, K = rows.shape
    E = layer[0].shape[0]
    if T * topk <= E:  # few slots: each with its own expert's weight
        w = _dequant(*(t[ids.reshape(-1)] for t in layer))
        return torch.bmm(rows.reshape(T * topk, 1, K), w).view(T, topk, -1)
    made = torch.matmul(rows.reshape(1, T * topk, K), _dequant(*layer))  # every row by every expert
    at = torch.arange(T * topk, device=rows.device)
    return made[ids.reshape(-1), at].view(T, topk, -1)


def _plain_layer(state):
    case, x = state["case"], state["x"]
    logits = torch.matmul(x.double(), state["router"].double().t())  # choices lie next to each other
    weights, ids = _plain_route(case, logits, state["bias"])
    both = _plain_product(x.float().unsqueeze(1).expand(-1, case["topk"], -1), state["gate_up"], ids)
    h = _silu(both[:, :, :case["inner"]]) * both[:, :, case["inner"]:]
    y = (_plain_product(h, state["down"], ids) * weights.unsqueeze(2)).sum(dim=1)
    if state["residual"] is not None:
        y = y + state["residual"].float()
    return y.to(x.dtype)


PLAIN = {"fused": _plain_fused, "norm": _plain_norm, "layer": _plain_layer}


# ---- The framework's operators.

def _framework(state):
    import w4a16_weight_only_amd as awq

    case = state["case"]
    if case["op"] == "fused":
        return awq.awq_gemm_fused(state["x"], *state["weight"], state["bias"], case["g"],
                                  activation=None if case["act"] == "none" else case["act"], gated=case["gated"],
                                  residual=state["residual"], scale=case["scale"])
    if case["op"] == "norm":
        return awq.awq_add_norm(state["x"], state["residual"], state["weight"], state["bias"], kind=case["kind"],
                                eps=EPS, gate=state["gate"], scale=case["scale"], post_weight=state["post_weight"],
                                post_bias=state["post_bias"], unit_offset=case["unit_offset"])
    return awq.awq_moe_layer(state["x"], state["router"], state["gate_up"], state["down"], case["topk"], case["g"],
                             score=case["score"], bias=state["bias"], groups=case["groups"],
                             topk_groups=case["topk_groups"], group_top=case["group_top"], scale=case["scale"],
                             residual=state["residual"])


def run(state):
    return _framework(state) if own else PLAIN[state["case"]["op"]](state)


# ---- The definition in 64 bits, apart from the plain form.

def _exact_weight(layer):
    """A packed weight [K, N] in 64 bits, one nibble of every word at a time."""
    qweight, qzeros, scales = layer
    K, words = qweight.shape
    w = torch.empty((K, words, 8), dtype=torch.float64, device=qweight.device)
    row_group = torch.arange(K, device=qweight.device) // (K // qzeros.shape[0])
    s = scales.double().view(scales.shape[0], words, 8)
    for nibble, column in enumerate((0, 2, 4, 6, 1, 3, 5, 7)):
        code = torch.bitwise_and(torch.bitwise_right_shift(qweight, 4 * nibble), 15).double()
        zero = torch.bitwise_and(torch.bitwise_right_shift(qzeros, 4 * nibble), 15).double()
        w[:, :, column] = (code - zero[row_group]) * s[row_group, :, column]
    return w.view(K, words * 8)


def _exact_activation(kind, v):
    if kind == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if kind == "silu":
        return v * torch.sigmoid(v)
    if kind == "gelu":
        return v * torch.special.ndtr(v)
    if kind == "gelu_tanh":  # (1 + tanh u) / 2 is the logistic function of 2 u
        return v * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))
    return v


def _exact_fused(state):
    case = state["case"]
    v = state["x"].double() @ _exact_weight(state["weight"])
    if state["bias"] is not None:
        v += state["bias"].double()
    if case["gated"]:
        first, second = v.split(case["N"], dim=1)
        v = _exact_activation(case["act"], first) * second
    else:
        v = _exact_activation(case["act"], v)
    v = case["scale"] * v
    return v if state["residual"] is None else state["residual"].double() + v


def _exact_norm(state):
    case = state["case"]

    def normed(v, weight, bias):
        spread, mean = torch.var_mean(v, dim=1, correction=0, keepdim=True)
        v = (v - mean) * torch.rsqrt(spread + EPS) if case["kind"] == "layer" else v * torch.rsqrt(spread + mean * mean + EPS)
        w = 1.0 + weight.double() if case["unit_offset"] else weight.double()
        return v * w if bias is None else torch.addcmul(bias.double(), v, w)

    x = state["x"].double()
    z = normed(x, state["post_weight"], state["post_bias"]) if case["post"] else x
    if state["gate"] is not None:
        B, H = state["gate"].shape
        z = (z.view(B, -1, H) * state["gate"].double().unsqueeze(1)).view(-1, H)
    r = torch.add(state["residual"].double(), z, alpha=case["scale"])
    return normed(r, state["weight"], state["bias"]), r


def _exact_choice(case, lg, bias):
    """(weights, ids) in numpy, from logits in 64 bits."""
    T, E = lg.shape
    if case["score"] == "softmax":
        e = np.exp(lg - lg.max(axis=1, keepdims=True))
        score = e / e.sum(axis=1, keepdims=True)
    else:
        score = np.where(lg >= 0, 1.0 / (1.0 + np.exp(-np.abs(lg))), np.exp(-np.abs(lg)) / (1.0 + np.exp(-np.abs(lg))))
    choice = score.copy() if bias is None else score + bias[None, :]
    G = case["groups"]
    if G > 1:
        best = -np.sort(-choice.reshape(T, G, E // G), axis=2)
        worth = best[:, :, :case["group_top"]].sum(axis=2)
        kept = np.argsort(-worth, axis=1, kind="stable")[:, :case["topk_groups"]]
        drop = np.ones((T, G), dtype=bool)
        np.put_along_axis(drop, kept, False, axis=1)
        choice[np.repeat(drop, E // G, axis=1)] = -np.inf
    ids = np.argsort(-choice, axis=1, kind="stable")[:, :case["topk"]]
    w = np.take_along_axis(score, ids, axis=1)
    return w / w.sum(axis=1, keepdims=True) * case["scale"], ids


def _exact_layer(state):
    case = state["case"]
    x = state["x"].double()
    logits = (x.unsqueeze(1) * state["router"].double().unsqueeze(0)).sum(dim=2)
    bias = None if state["bias"] is None else state["bias"].double().cpu().numpy()
    weights, ids = _exact_choice(case, logits.cpu().numpy(), bias)
    y = torch.zeros_like(x) if state["residual"] is None else state["residual"].double()
    for e in np.unique(ids):
        token, j = (torch.from_numpy(a).to(x.device) for a in np.nonzero(ids == e))
        part = lambda layer: _exact_weight([t[int(e)] for t in layer])  # noqa: E731
        gate, up = (x[token] @ part(state["gate_up"])).split(case["inner"], dim=1)
        made = (gate * torch.sigmoid(gate) * up) @ part(state["down"])
        y.index_add_(0, token, made * torch.from_numpy(weights).to(x.device)[token, j][:, None])
    return y


def exact(case, seed):
    return {"fused": _exact_fused, "norm": _exact_norm, "layer": _exact_layer}[case["op"]](prepare(case, seed))
