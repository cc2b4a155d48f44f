"""Measured cases of two operators that stand next to the quantized expert layer.

* routing to experts by scores: softmax or sigmoid scores of the router's logits, a bias that
  steers the choice only, a choice limited to the best groups of experts, the k best experts,
  their (renormalised, scaled) scores as weights, and the permutation that the expert products
  read (``moe_route_scored``);
* a dense product with packed weights: out = [residual +] [mul *] act(x.W + bias), for the
  projections of a model that are no experts (attention output, dense feed-forward layers, the
  two halves of a gated one), in the expert layer's own packed format (``moe_linear_forward``).

``run`` computes them in elementary torch operations (32 bits; the routing's choice in 64, where
two experts' values may lie next to each other) or, where ``own`` is true, by the library.
"""
import math

import numpy as np
import torch

own = False

TERNARY, INT2, INT3 = 1, 2, 3
LEVELS = {TERNARY: 3, INT2: 4, INT3: 8}
OFFSET = {TERNARY: 1.0, INT2: 1.5, INT3: 3.5}
ACTS = ("none", "silu", "gelu", "gelu_tanh", "relu", "relu2", "sigmoid")


# ------------------------------------------------------------------------------- the cases
def _route(name, T, E, k, score, groups=1, topk_groups=1, group_top=1, bias=False, renorm=True,
           scale=1.0, skew=0.0, masked=0):
    c = {"op": "route", "T": T, "E": E, "k": k, "score": score, "groups": groups,
         "topk_groups": topk_groups, "group_top": group_top, "bias": bias, "renorm": renorm,
         "scale": scale, "skew": skew, "masked": masked}
    return {"name": name, **c} if name else c


def _linear(name, T, K, N, q, act="none", bias=False, mul=False, residual=False, pad=0):
    c = {"op": "linear", "T": T, "K": K, "N": N, "q": q, "act": act, "bias": bias, "mul": mul,
         "residual": residual, "pad": pad}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one token being generated: latency alone counts
        _route("route_token", 1, 256, 8, "sigmoid", 8, 4, 2, bias=True, scale=2.5),
        # a decode batch of the layer's eight tokens, no groups, hot experts
        _route("route_batch", 8, 256, 8, "softmax", skew=1.1),
        # a ragged chunk of a prompt, group sizes that are no power of two, a few pruned experts
        _route("route_ragged", 1237, 160, 6, "softmax", 8, 3, 1, renorm=False, scale=16.0,
               masked=9),
        # a whole prompt, with groups and a balance bias
        _route("route_prompt", 8192, 256, 8, "sigmoid", 8, 4, 2, bias=True, scale=2.5),
        # the longest prompt, skewed to hot experts, weights renormalised
        _route("route_long", 16384, 256, 8, "softmax", skew=1.2),
        # one token through an output projection onto the residual stream
        _linear("linear_token", 1, 4096, 4096, INT2, residual=True),
        # a decode batch through the gate half of a gated feed-forward layer, the up half given
        _linear("linear_batch", 8, 4096, 2048, INT3, "silu", mul=True),
        # a short prompt, ragged in rows and in columns, rows padded apart
        _linear("linear_chunk", 77, 4096, 2064, INT2, "gelu", bias=True, pad=8),
        # a few hundred tokens, an odd number of k-blocks
        _linear("linear_few_hundred", 300, 2176, 4096, TERNARY, "relu2", bias=True),
        # a prompt through the gate half of a gated feed-forward layer
        _linear("linear_prompt", 8192, 4096, 2048, INT2, "silu", mul=True),
        # the same prompt through ternary weights, back onto the residual stream
        _linear("linear_prompt_down", 8192, 2048, 4096, TERNARY, residual=True),
        # the longest prompt through a square projection
        _linear("linear_long", 16384, 4096, 4096, INT3, residual=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.45:
        while True:
            T, E = _log(rng, 1, 16384), rng.choice([8, 40, 64, 96, 128, 160, 256, 384, 512, 1024])
            groups = rng.choice([g for g in (1, 1, 2, 4, 5, 8, 16) if E % g == 0 and E // g >= 4])
            tg = rng.randint(1, groups)
            k = rng.randint(1, min(32, tg * (E // groups)))
            if T * E <= 16384 * 256 and T * k <= 16384 * 8:
                break
        return _route(None, T, E, k, rng.choice(["softmax", "sigmoid"]), groups, tg,
                      rng.choice([1, 2]), rng.random() < 0.5, rng.random() < 0.7,
                      rng.choice([1.0, 2.5, 16.0]), rng.choice([0.0, 0.0, 1.2]),
                      rng.choice([0, 0, E // 16]))
    while True:
        T = _log(rng, 1, 16384)
        K, N = 128 * _log(rng, 1, 64), 16 * _log(rng, 1, 512)
        if T * K * N <= 16384 * 4096 * 4096 and (T + N) * K <= (16384 + 4096) * 4096:
            break
    return _linear(None, T, K, N, rng.choice([TERNARY, INT2, INT3]), rng.choice(ACTS),
                   rng.random() < 0.5, rng.random() < 0.4, rng.random() < 0.5,
                   rng.choice([0, 0, 8, 72]))


# ------------------------------------------------------------------------------ the inputs
def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _rows(g, T, width, pad):
    """bf16 rows of N(0, 1), `pad` values apart from one another."""
    return _normal(g, T, width + pad).to(torch.bfloat16)[:, :width]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": dict(case)}
    if case["op"] == "route":
        T, E = case["T"], case["E"]
        logits = _normal(g, T, E)
        if case["skew"]:  # a logit bias ln p_e, p_e by a power law over the experts in some order
            rank = torch.randperm(E, generator=g, device="cuda").float()
            logits -= case["skew"] * torch.log(rank + 1.0)
        if case["masked"]:  # experts that were taken out of the model
            logits[:, torch.randperm(E, generator=g, device="cuda")[:case["masked"]]] = -math.inf
        s["logits"] = logits
        s["bias"] = 0.1 * _normal(g, E) if case["bias"] else None
    else:
        T, K, N, q, pad = (case[n] for n in ("T", "K", "N", "q", "pad"))
        s["codes"] = torch.randint(0, LEVELS[q], (N, K), generator=g, device="cuda",
                                   dtype=torch.uint8)
        s["scales"] = (0.05 * _normal(g, N, K // 32)).abs().to(torch.float16)
        s["x"] = _rows(g, T, K, pad)
        s["bias"] = 0.5 * _normal(g, N) if case["bias"] else None
        s["mul"] = _rows(g, T, N, pad) if case["mul"] else None
        s["residual"] = _rows(g, T, N, pad) if case["residual"] else None
    if own:  # the handle, workspace and output buffers that a program keeps
        s.update(_own_route(s) if case["op"] == "route" else _own_linear(s))
    return s


# -------------------------------------------------------------------------- the plain forms
def _plain_route(s):
    c, l = s["case"], s["logits"].double()
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    out = l == -math.inf
    if c["score"] == "softmax":
        score = torch.exp(l - l.max(1, keepdim=True).values)
        score = score / score.sum(1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-l))
    choice = score if s["bias"] is None else score + s["bias"].double()
    choice = choice.masked_fill(out, -math.inf)
    if G > 1:
        best = choice.view(T, G, E // G).sort(dim=2, descending=True).values[:, :, :c["group_top"]]
        order = best.sum(2).sort(dim=1, descending=True, stable=True).indices[:, :c["topk_groups"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, order, True)
        # a masked expert comes after all others of its group, but before those of other groups
        choice = choice.clamp(min=torch.finfo(torch.float64).min)
        choice = choice.masked_fill(~keep.repeat_interleave(E // G, 1), -math.inf)
    ids = choice.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    by_expert, rows = ids.reshape(-1).sort(dim=0, stable=True)
    offsets = torch.searchsorted(by_expert, torch.arange(E + 1, device=l.device))
    inv = torch.empty_like(rows)
    inv[rows] = torch.arange(T * k, device=l.device)
    whole = {"ids": ids, "counts": offsets[1:] - offsets[:-1], "offsets": offsets,
             "perm_tok": rows // k, "inv_row": inv.view(T, k)}
    return {"weights": (w * c["scale"]).float(), **{n: v.to(torch.int32) for n, v in whole.items()}}


def _act(name, v):
    if name == "silu":
        return v / (1.0 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v / math.sqrt(2.0)))
    if name == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    if name == "relu":
        return torch.clamp(v, min=0.0)
    if name == "relu2":
        return torch.clamp(v, min=0.0) ** 2
    if name == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-v))
    return v


def _plain_linear(s):
    c = s["case"]
    K, N = c["K"], c["N"]
    w = (s["codes"].float() - OFFSET[c["q"]]).view(N, K // 32, 32) * s["scales"].float()[:, :, None]
    v = s["x"].float() @ w.view(N, K).t()
    if s["bias"] is not None:
        v = v + s["bias"]
    v = _act(c["act"], v)
    if s["mul"] is not None:
        v = v * s["mul"].float()
    if s["residual"] is not None:
        v = v + s["residual"].float()
    return v.to(torch.bfloat16)


# ---------------------------------------------------------------------- the library's calls
def _own_route(s):
    import bit_quantized_moe_router_amd as bq

    c = s["case"]
    layer = bq.make_layer(256, 128, c["E"], c["k"], 0, (2, 2, 2), None, 0)
    scoring = bq.make_scoring(bq.MOE_SCORE_SOFTMAX if c["score"] == "softmax" else
                              bq.MOE_SCORE_SIGMOID, n_groups=c["groups"],
                              topk_groups=c["topk_groups"], group_top=c["group_top"],
                              renorm=c["renorm"], scale=c["scale"], choice_bias=s["bias"])
    return {"bq": bq, "layer": layer, "scoring": scoring,
            "routing": bq.alloc_routing(c["T"], c["E"], c["k"], logits=s["logits"]),
            "ws": bq.alloc_workspace(layer, c["T"])}


def _own_linear(s):
    import bit_quantized_moe_router_amd as bq

    c = s["case"]
    blob = bq.moe_pack_weights(c["q"], s["codes"].cpu().numpy(),
                               s["scales"].cpu().numpy().view(np.uint16))
    act = {"none": bq.MOE_ACT_NONE, "silu": bq.MOE_ACT_SILU, "gelu": bq.MOE_ACT_GELU,
           "gelu_tanh": bq.MOE_ACT_GELU_TANH, "relu": bq.MOE_ACT_RELU, "relu2": bq.MOE_ACT_RELU2,
           "sigmoid": bq.MOE_ACT_SIGMOID}[c["act"]]
    lin = bq.make_linear(c["K"], c["N"], c["q"], torch.from_numpy(blob).cuda(), bias=s["bias"],
                         act=act)
    out = torch.empty(c["T"], c["N"], dtype=torch.bfloat16, device="cuda")
    return {"bq": bq, "lin": lin, "out": out, "ws": bq.alloc_linear_workspace(lin, c["T"])}


def run(state):
    s = state
    if s["case"]["op"] == "route":
        if not own:
            return _plain_route(s)
        r = s["routing"]
        s["bq"].moe_route_scored(s["layer"], s["scoring"], None, s["case"]["T"],
                                 s["bq"].MOE_LOGITS_GIVEN, r, s["ws"])
        return {"ids": r.topk_ids, "weights": r.topk_w, "counts": r.counts, "offsets": r.offsets,
                "perm_tok": r.perm_tok, "inv_row": r.inv_row}
    if not own:
        return _plain_linear(s)
    s["bq"].moe_linear_forward(s["lin"], s["x"], s["case"]["T"], s["out"], s["ws"], mul=s["mul"],
                               residual=s["residual"])
    return s["out"]


# ------------------------------------------------------------------------------- accounting
def work(case):
    T = case["T"]
    if case["op"] == "route":
        E, k = case["E"], case["k"]
        # logits and bias in; ids, weights, row maps, counts and offsets out
        return {"bytes": 4 * T * E + 4 * E * case["bias"] + 16 * T * k + 8 * E + 4,
                "flops": 4 * T * E}
    K, N = case["K"], case["N"]
    bits = 3 if case["q"] == INT3 else 2
    packed = K * N * bits // 8 + K * N // 32 * 2
    rows = 2 * T * K + 2 * T * N * (1 + case["mul"] + case["residual"])
    return {"bytes": packed + rows + 4 * N * case["bias"], "flops": 2 * T * K * N}


# ------------------------------------------------------------------ the definitions, 64 bits
def _exact_route(case, s):
    """Row by row of the definition, on the host: ranks by (value down, index up)."""
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    l = s["logits"].cpu().numpy().astype(np.float64)
    gone = np.isneginf(l)
    if case["score"] == "softmax":
        e = np.exp(l - l.max(axis=1)[:, None])
        p = e / e.sum(axis=1)[:, None]
    else:
        p = 1.0 / (1.0 + np.exp(-l))
    b = np.zeros(E) if s["bias"] is None else s["bias"].cpu().numpy().astype(np.float64)
    v = np.where(gone, -np.inf, p + b)
    if G > 1:
        gv = np.sort(v.reshape(T, G, -1), axis=2)[:, :, -case["group_top"]:].sum(axis=2)
        place = np.argsort(np.argsort(-gv, axis=1, kind="stable"), axis=1)
        second = np.repeat(place >= case["topk_groups"], E // G, axis=1)
    else:
        second = np.zeros((T, E), bool)
    # last key first: the group out of the choice, then the value, then the index
    ids = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), -v, second), axis=1)[:, :k]
    w = np.take_along_axis(p, ids, axis=1)
    if case["renorm"]:
        w = w / w.sum(axis=1)[:, None]
    flat = ids.reshape(-1)
    rows = np.argsort(flat, kind="stable")
    inv = np.empty(T * k, np.int64)
    inv[rows] = np.arange(T * k)
    counts = np.bincount(flat, minlength=E)
    ints = {"ids": ids, "counts": counts, "offsets": np.concatenate([[0], np.cumsum(counts)]),
            "perm_tok": rows // k, "inv_row": inv.reshape(T, k)}
    return {"weights": w * case["scale"], **{n: np.asarray(a, np.int32) for n, a in ints.items()}}


def _exact_linear(case, s):
    """64 bits throughout, a block of columns at a time."""
    T, K, N = case["T"], case["K"], case["N"]
    x = s["x"].double()
    out = torch.empty(T, N, dtype=torch.float64, device="cuda")
    for n0 in range(0, N, 1024):
        cols = slice(n0, min(N, n0 + 1024))
        u = s["codes"][cols].double()
        step = s["scales"][cols].double().repeat_interleave(32, dim=1)
        out[:, cols] = torch.mm(x, ((u - OFFSET[case["q"]]) * step).t().contiguous())
    if s["bias"] is not None:
        out += s["bias"].double()
    a = case["act"]
    if a in ("silu", "sigmoid"):
        sig = torch.sigmoid(out)
        out = out * sig if a == "silu" else sig
    elif a == "gelu":
        out = out * 0.5 * torch.erfc(-out * math.sqrt(0.5))
    elif a == "gelu_tanh":
        out = out * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (out + 0.044715 * out ** 3))
    elif a in ("relu", "relu2"):
        out = torch.where(out > 0, out, torch.zeros_like(out)) ** (2 if a == "relu2" else 1)
    if s["mul"] is not None:
        out *= s["mul"].double()
    if s["residual"] is not None:
        out += s["residual"].double()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_route(case, s) if case["op"] == "route" else _exact_linear(case, s)
