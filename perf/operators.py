"""The routed-expert operators' measured cases: their inputs, their plain form in elementary
torch operations, and their definition in 64 bits.

Four operators make up a routed-expert layer on AWQ GEMM-layout weights:

  route     logits [T, E] -> the topk experts of each token and their weights
  gate_up   x [T, K] -> h [T * topk, I] = silu(x . Wg[e]) * (x . Wu[e]), Wg and Wu the two halves
            of the expert's [K, 2 I] weight
  down      h [T * topk, K] -> y [T, N] = sum over a token's slots of weight * (h[slot] . W[e])
  mlp       gate_up and down in one call

`own` false: the plain form. `own` true: the framework's entry points.
"""
import math

import numpy as np
import torch

own = False

# Column j of a packed word sits in nibble INVERSE[j].
INVERSE = (0, 4, 1, 5, 2, 6, 3, 7)
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def _route(name, T, E, topk, dtype, score, bias=False, groups=1, topk_groups=1, group_top=1, renormalize=True,
           scale=1.0, masked=False):
    return dict(name=name, op="route", T=T, E=E, topk=topk, dtype=dtype, score=score, bias=bias, groups=groups,
                topk_groups=topk_groups, group_top=group_top, renormalize=renormalize, scale=scale, masked=masked)


def _experts(name, op, T, E, topk, K, inner, N, g, dtype):
    return dict(name=name, op=op, T=T, E=E, topk=topk, K=K, inner=inner, N=N, g=g, dtype=dtype)


def listed():
    return [
        # One decoding token through a layer of 64 experts: latency alone.
        _route("route_token", 1, 64, 8, "f16", "softmax"),
        # A decoding batch of a large layer: sigmoid scores, a balancing bias, 4 of 8 groups kept
        # by their two best experts, renormalised and scaled weights.
        _route("route_groups", 512, 256, 8, "bf16", "sigmoid", bias=True, groups=8, topk_groups=4, group_top=2,
               scale=2.5),
        # A long prompt, scores kept in 32 bits.
        _route("route_prompt", 16384, 128, 8, "f32", "softmax"),
        # One decoding token of the 8-expert layer (4096 -> 14336): two experts' weights are read.
        _experts("gate_up_token", "gate_up", 1, 8, 2, 4096, 14336, 0, 128, "f16"),
        # An odd decoding batch of a many-expert layer: about six rows per expert.
        _experts("gate_up_batch", "gate_up", 45, 64, 8, 2048, 1408, 0, 64, "bf16"),
        # A prompt through the 8-expert layer: matrix products of about 256 rows per expert.
        _experts("gate_up_prompt", "gate_up", 1024, 8, 2, 4096, 14336, 0, 128, "f16"),
        # The second product for one token of the many-expert layer.
        _experts("down_token", "down", 1, 64, 8, 1408, 0, 2048, 128, "bf16"),
        # An odd batch on the long axis of the 8-expert layer, one quantization group over it.
        _experts("down_batch", "down", 19, 8, 2, 14336, 0, 4096, -1, "f16"),
        # A prompt through the many-expert layer, the smallest groups.
        _experts("down_prompt", "down", 1536, 64, 8, 1408, 0, 2048, 32, "bf16"),
        # A whole routed layer for one token, for a decoding batch and for a prompt.
        _experts("mlp_token", "mlp", 1, 64, 8, 2048, 1408, 2048, 128, "f16"),
        _experts("mlp_batch", "mlp", 16, 8, 2, 4096, 14336, 4096, 128, "bf16"),
        _experts("mlp_prompt", "mlp", 2048, 64, 8, 2048, 1408, 2048, 64, "f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "gate_up", "down", "mlp"))
    if op == "route":
        groups = rng.choice((1, 1, 4, 8))
        E = groups * rng.randint(4, 256 // groups)
        topk_groups = rng.randint(1, groups)
        topk = min(rng.randint(1, 8), topk_groups * (E // groups))
        c = _route("", _log(rng, 1, 8192), E, topk, rng.choice(("f16", "bf16", "f32")),
                   rng.choice(("softmax", "sigmoid")), bias=rng.random() < 0.5, groups=groups,
                   topk_groups=topk_groups, group_top=rng.choice((1, 2)), renormalize=rng.random() < 0.7,
                   scale=rng.choice((1.0, 2.5)), masked=rng.random() < 0.3)
    else:
        E, topk = rng.choice(((1, 1), (8, 2), (16, 4), (60, 4), (64, 8), (128, 8)))
        g = rng.choice((32, 64, 128, 128, -1))
        step = 32 if g == -1 else g
        size = lambda lo, hi: max(step, _log(rng, lo, hi) // step * step)  # noqa: E731
        odd = lambda lo, hi: _log(rng, lo, hi) // 32 * 32  # noqa: E731  (columns need not be whole groups)
        K = size(512, 4096)
        inner = 0 if op == "down" else odd(256, 4096) if op == "gate_up" else size(256, 4096)
        N = 0 if op == "gate_up" else odd(512, 4096)
        c = _experts("", op, 1, E, topk, K, inner, N, g, rng.choice(("f16", "bf16")))
        per_slot = max(1, _weights(c))
        c["T"] = _log(rng, 1, max(1, min(2048, 200_000_000_000 // (2 * per_slot * topk))))
    del c["name"]
    return c


def _weights(case):
    """Weights of one expert that the case's operator multiplies by."""
    K, inner, N = case["K"], case["inner"], case["N"]
    return {"gate_up": 2 * K * inner, "down": K * N, "mlp": 2 * K * inner + inner * N}[case["op"]]


def work(case):
    T, E, topk = case["T"], case["E"], case["topk"]
    if case["op"] == "route":
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": T * E * size + (4 * E if case["bias"] else 0) + T * topk * 8, "flops": 4 * T * E}
    K, inner, N, g = case["K"], case["inner"], case["N"], case["g"]
    slots = T * topk
    active = E * (1.0 - (1.0 - topk / E) ** T)  # experts with a slot, for even routing

    def layer(k, n):  # packed weights, zeros and scales
        return k * n // 2 + (k // (k if g == -1 else g)) * (n // 2 + 2 * n)

    if case["op"] == "gate_up":
        moved = active * layer(K, 2 * inner) + 2 * T * K + 4 * slots + 2 * slots * inner
    elif case["op"] == "down":
        moved = active * layer(K, N) + 2 * slots * K + 8 * slots + 2 * T * N
    else:
        moved = active * (layer(K, 2 * inner) + layer(inner, N)) + 2 * T * K + 8 * slots + 2 * T * N
    return {"bytes": int(moved), "flops": 2 * slots * _weights(case)}


# ---- Inputs.

def _layer(gen, E, K, N, g):
    """One stacked weight: uniform codes and zeros, scales that keep a product's size near its
    input's (codes less zeros have a spread of about 6.5)."""
    G = 1 if g == -1 else K // g
    words = lambda *shape: torch.randint(-(1 << 31), 1 << 31, shape, dtype=torch.int32, device="cuda", generator=gen)  # noqa: E731
    scales = torch.rand((E, G, N), device="cuda", generator=gen).add_(0.5).mul_(1.0 / (6.5 * math.sqrt(K)))
    return words(E, K, N // 8), words(E, G, N // 8), scales.half()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, device="cuda", generator=gen)  # noqa: E731
    T, E, topk = case["T"], case["E"], case["topk"]
    # Router outputs: some experts are liked by more tokens than others.
    logits = 1.5 * normal(T, E) + 0.5 * normal(1, E)
    if case["op"] == "route":
        logits = logits.to(TYPES[case["dtype"]])
        if case["masked"]:  # experts that are switched off for some tokens; now and then all of them
            off = torch.rand((T, E), device="cuda", generator=gen) < 0.3
            off |= torch.rand((T, 1), device="cuda", generator=gen) < 0.02
            logits.masked_fill_(off, -math.inf)
        bias = 0.2 * normal(E) if case["bias"] else None
        return dict(case=case, logits=logits, bias=bias)
    top = logits.topk(topk, dim=1)
    state = dict(case=case, ids=top.indices.to(torch.int32).contiguous(),
                 weights=top.values.softmax(dim=1).contiguous())
    K, inner, N, g = case["K"], case["inner"], case["N"], case["g"]
    dtype = TYPES[case["dtype"]]
    if case["op"] == "down":
        state["x"] = normal(T * topk, K).to(dtype)
        state["down"] = _layer(gen, E, K, N, g)
    else:
        state["x"] = normal(T, K).to(dtype)
        state["gate_up"] = _layer(gen, E, K, 2 * inner, g)
        if case["op"] == "mlp":
            state["down"] = _layer(gen, E, inner, N, g)
    return state


# ---- The plain form.

def _plain_route(case, logits, bias):
    T, E = logits.shape
    off = logits == -math.inf
    lg = logits.double()  # scores in 64 bits: experts a rounding apart must come out in order
    if case["score"] == "softmax":
        top = lg.amax(dim=1, keepdim=True)
        p = torch.exp(lg - torch.where(top == -math.inf, 0.0, top))
        score = p / p.sum(dim=1, keepdim=True).clamp_min(1e-300)
    else:
        score = 1.0 / (1.0 + torch.exp(-lg))
    choice = score if bias is None else score + bias.double()
    choice = choice.masked_fill(off, -math.inf)
    G = case["groups"]
    if G > 1:
        best = choice.view(T, G, E // G).sort(dim=2, descending=True).values
        worth = best[:, :, 0]
        if case["group_top"] == 2 and E // G > 1:
            second = best[:, :, 1]
            worth = worth + torch.where(second == -math.inf, 0.0, second)
        rank = worth.sort(dim=1, descending=True, stable=True).indices
        keep = torch.zeros((T, G), dtype=torch.bool, device=logits.device)
        keep.scatter_(1, rank[:, :case["topk_groups"]], True)
        choice = choice.masked_fill(~keep.repeat_interleave(E // G, dim=1), -math.inf)
    value, ids = choice.sort(dim=1, descending=True, stable=True)
    value, ids = value[:, :case["topk"]], ids[:, :case["topk"]]
    none = value == -math.inf
    w = score.gather(1, ids).masked_fill(none, 0.0)
    if case["renormalize"]:
        w = w / w.sum(dim=1, keepdim=True).clamp_min(1e-300)
    return (w * case["scale"]).float(), ids.masked_fill(none, -1).int()


def _dequant(qweight, qzeros, scales):
    """[B, K, N] in 32 bits: (code - zero) * scale."""
    shift = 4 * torch.tensor(INVERSE, dtype=torch.int32, device=qweight.device)
    B, K, words = qweight.shape
    G = qzeros.shape[1]
    q = ((qweight.unsqueeze(-1) >> shift) & 15).view(B, G, K // G, words * 8)
    z = ((qzeros.unsqueeze(-1) >> shift) & 15).view(B, G, 1, words * 8)
    return ((q - z).float() * scales.float().unsqueeze(2)).view(B, K, words * 8)


def _plain_product(rows, layer, ids):
    """rows [S, K] (32 bits), slot s by expert ids[s] -> [S, N] (32 bits)."""
    S, E = ids.numel(), layer[0].shape[0]
    ids = ids.reshape(-1).long()
    if S <= E:  # few slots: each with its own expert's weight
        w = _dequant(*(t[ids] for t in layer))
        return torch.bmm(rows.unsqueeze(1), w).squeeze(1)
    order = ids.argsort(stable=True)
    of = ids[order]
    count = torch.bincount(ids, minlength=E)
    place = torch.arange(S, device=ids.device) - (count.cumsum(0) - count)[of]
    padded = torch.zeros((E, int(count.max()), rows.shape[1]), device=rows.device)
    padded[of, place] = rows[order]
    made = torch.bmm(padded, _dequant(*layer))
    out = torch.empty((S, made.shape[2]), device=rows.device)
    out[order] = made[of, place]
    return out


def _plain_gate_up(x, layer, ids):
    topk = ids.shape[1]
    both = _plain_product(x.float().repeat_interleave(topk, dim=0), layer, ids)
    inner = both.shape[1] // 2
    gate = both[:, :inner]
    return gate / (1.0 + torch.exp(-gate)) * both[:, inner:]


def _plain_down(h, layer, ids, weights):
    T, topk = ids.shape
    return (_plain_product(h, layer, ids).view(T, topk, -1) * weights.unsqueeze(2)).sum(dim=1)


def _plain(state):
    case = state["case"]
    if case["op"] == "route":
        return _plain_route(case, state["logits"], state["bias"])
    x = state["x"]
    if case["op"] == "gate_up":
        return _plain_gate_up(x, state["gate_up"], state["ids"]).to(x.dtype)
    h = x.float() if case["op"] == "down" else _plain_gate_up(x, state["gate_up"], state["ids"])
    return _plain_down(h, state["down"], state["ids"], state["weights"]).to(x.dtype)


# ---- The framework's operators.

def _framework(state):
    import w4a16_weight_only_amd as awq

    case = state["case"]
    if case["op"] == "route":
        return awq.awq_moe_route(state["logits"], case["topk"], score=case["score"], bias=state["bias"],
                                 groups=case["groups"], topk_groups=case["topk_groups"],
                                 group_top=case["group_top"], renormalize=case["renormalize"], scale=case["scale"])
    if case["op"] == "gate_up":
        return awq.awq_moe_gate_up(state["x"], *state["gate_up"], state["ids"], case["g"])
    if case["op"] == "down":
        return awq.awq_moe_down(state["x"], *state["down"], state["ids"], state["weights"], case["g"])
    return awq.awq_moe_mlp(state["x"], state["gate_up"], state["down"], state["ids"], state["weights"], case["g"])


def run(state):
    return _framework(state) if own else _plain(state)


# ---- The definition in 64 bits, apart from the plain form.

def _exact_route(case, logits, bias):
    lg = logits.double().cpu().numpy()
    T, E = lg.shape
    off = np.isneginf(lg)
    with np.errstate(over="ignore", under="ignore", invalid="ignore"):
        if case["score"] == "softmax":
            top = lg.max(axis=1, keepdims=True)
            e = np.exp(np.where(off, -np.inf, lg - np.where(np.isneginf(top), 0.0, top)))
            total = e.sum(axis=1, keepdims=True)
            score = np.divide(e, total, out=np.zeros_like(e), where=total > 0)
        else:
            score = np.where(lg >= 0, 1.0 / (1.0 + np.exp(-lg)), np.exp(lg) / (1.0 + np.exp(lg)))
    choice = score.copy() if bias is None else score + bias.double().cpu().numpy()[None, :]
    choice[off] = -np.inf
    G, per = case["groups"], E // case["groups"]
    if G > 1:
        parts = choice.reshape(T, G, per)
        best = -np.sort(-parts, axis=2)
        worth = best[:, :, 0].copy()
        if case["group_top"] == 2 and per > 1:
            worth += np.where(np.isneginf(best[:, :, 1]), 0.0, best[:, :, 1])
        kept = np.argsort(-worth, axis=1, kind="stable")[:, :case["topk_groups"]]
        drop = np.ones((T, G), dtype=bool)
        np.put_along_axis(drop, kept, False, axis=1)
        choice[np.repeat(drop, per, axis=1)] = -np.inf
    ids = np.argsort(-choice, axis=1, kind="stable")[:, :case["topk"]]
    none = np.isneginf(np.take_along_axis(choice, ids, axis=1))
    w = np.where(none, 0.0, np.take_along_axis(score, ids, axis=1))
    if case["renormalize"]:
        total = w.sum(axis=1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    return torch.from_numpy(w * case["scale"]), torch.from_numpy(np.where(none, -1, ids).astype(np.int32))


def _exact_weight(layer, e):
    """Expert e's [K, N] weight in 64 bits, one nibble of every word at a time."""
    qweight, qzeros, scales = (t[e] for t in layer)
    K, words = qweight.shape
    w = torch.empty((K, words, 8), dtype=torch.float64, device=qweight.device)
    row_group = torch.arange(K, device=qweight.device) // (K // qzeros.shape[0])
    s = scales.double().view(scales.shape[0], words, 8)
    for nibble, column in enumerate((0, 2, 4, 6, 1, 3, 5, 7)):
        code = torch.bitwise_and(torch.bitwise_right_shift(qweight, 4 * nibble), 15).double()
        zero = torch.bitwise_and(torch.bitwise_right_shift(qzeros, 4 * nibble), 15).double()
        w[:, :, column] = (code - zero[row_group]) * s[row_group, :, column]
    return w.view(K, words * 8)


def _exact_experts(case, state):
    ids, x = state["ids"], state["x"].double()
    T, topk = ids.shape
    down = "down" in state
    out = torch.zeros((T, case["N"]) if down else (T * topk, case["inner"]), dtype=torch.float64, device=x.device)
    for e in range(case["E"]):
        token, j = torch.nonzero(ids == e, as_tuple=True)
        if token.numel() == 0:
            continue
        slot = token * topk + j
        v = x[slot] if case["op"] == "down" else x[token]
        if case["op"] != "down":
            both = v @ _exact_weight(state["gate_up"], e)
            gate, up = both.split(case["inner"], dim=1)
            v = gate * torch.sigmoid(gate) * up
        if down:
            out.index_add_(0, token, (v @ _exact_weight(state["down"], e)) * state["weights"][token, j].double()[:, None])
        else:
            out[slot] = v
    return out


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(case, state["logits"], state["bias"])
    return _exact_experts(case, state)
