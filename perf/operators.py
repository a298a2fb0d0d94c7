"""The operators at the edges of a routed-expert layer: what is timed, their plain forms and their exact values.

  select    strata_moe_select: routing from logits (softmax or sigmoid scores, balance bias, groups, top-k)
  norm      strata_moe_norm: the norm before a block
  edge      strata_moe_combine_norm: weighted sum of the experts' outputs, norm after the block, gates,
            scaled residual, and the next block's norm
  adapters  strata_moe_adapters: low-rank adapters of many requests beside a shared projection

The plain forms are elementary torch operations; with ``own`` set, run() makes the library's calls.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
F32_MAX = float(np.finfo(np.float32).max)
CLAMP = 2.0 ** -14  # lower clamp of the sum that renormalises the weights
MASKED_ROWS = 64    # of this many rows one has experts that are not available


# ------------------------------------------------------------------------------------------------
# Cases
# ------------------------------------------------------------------------------------------------
def select(T, E, k, score, groups=1, keep=1, group_sum=1, bias=False, renorm=True, scale=1.0, type="f32", **name):
    return dict(name, op="select", T=T, E=E, k=k, score=score, groups=groups, keep=keep, group_sum=group_sum, bias=bias,
                renorm=renorm, scale=scale, type=type)


def norm(T, n, x, out, pad=0, **name):
    return dict(name, op="norm", T=T, n=n, x=x, out=out, pad=pad)


def edge(T, n, parts, part, x, next, post=True, channel=True, token="none", residual=1.0, block=1.0, **name):
    return dict(name, op="edge", T=T, n=n, parts=parts, part=part, x=x, next=next, post=post, channel=channel, token=token,
                residual=residual, block=block)


def adapters(T, segments, count, rank, d_in, d_out, x, y, ragged=True, **name):
    return dict(name, op="adapters", T=T, segments=segments, count=count, rank=rank, d_in=d_in, d_out=d_out, x=x, y=y,
                ragged=ragged)


def listed():
    return [
        # one decoded token, the layer's own 512 experts and top-10: latency alone
        select(1, 512, 10, "softmax", name="select decode"),
        # a full prefill chunk with sigmoid scores, a balance bias and 4 of 16 groups kept
        select(8192, 512, 10, "sigmoid", groups=16, keep=4, group_sum=2, bias=True, scale=2.5, name="select prefill groups"),
        # a ragged chunk of a smaller layer: 160 experts in 8 groups, bf16 logits (many ties), weights not renormalised
        select(1237, 160, 6, "softmax", groups=8, keep=3, renorm=False, type="bf16", name="select ragged bf16"),
        # the verify window's input norm
        norm(4, 2560, "f32", "f32", name="norm verify"),
        # a full chunk's input norm, the stream in fp32 and the block's input in bf16
        norm(8192, 2560, "f32", "bf16", name="norm prefill"),
        # after one token's ten experts: combine, norm, gates, residual, the next layer's norm
        edge(1, 2560, 10, "f32", "f32", "f32", token="sigmoid", residual=0.9, name="edge decode"),
        # the same for a 2,048-token chunk
        edge(2048, 2560, 10, "f32", "f32", "f32", token="sigmoid", residual=0.9, name="edge prefill"),
        # after a whole layer call (its one fp32 output a token), the stream in bf16
        edge(8192, 2560, 1, "f32", "bf16", "bf16", block=0.5, name="edge prefill bf16"),
        # one token of one request, an adapter beside the router's projection
        adapters(1, 1, 4, 16, 2560, 512, "f32", "f32", name="adapters router decode"),
        # 64 requests decoding one token each, an adapter of their own each, beside the block
        adapters(64, 64, 64, 16, 2560, 2560, "bf16", "bf16", ragged=False, name="adapters decode"),
        # ragged prompts of 24 requests that share 12 adapters, fp32 activations
        adapters(2048, 24, 12, 32, 2560, 2560, "f32", "f32", name="adapters ragged f32"),
        # a full chunk of 32 prompts, rank 64
        adapters(8192, 32, 32, 64, 2560, 2560, "bf16", "bf16", name="adapters prefill"),
    ]


def spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("select", "select", "norm", "edge", "adapters", "adapters"))
    T = spread(rng, 1, 8192)
    if op == "select":
        groups = rng.choice((1, 1, 4, 8, 16))
        E = groups * spread(rng, max(2, 16 // groups), 512 // groups)
        keep = 1 if groups == 1 else rng.randint(1, groups)
        k = rng.randint(1, min(16, keep * (E // groups)))
        return select(T, E, k, rng.choice(("softmax", "sigmoid")), groups, keep, rng.choice((1, 2)), rng.random() < 0.5,
                      rng.random() < 0.7, rng.choice((1.0, 2.5)), rng.choice(("f32", "f32", "bf16", "f16")))
    kinds = ("f32", "bf16", "f16")
    if op == "norm":
        n = spread(rng, 64, 8192)
        return norm(min(T, 8192 * 2560 // n), n, rng.choice(kinds), rng.choice(kinds), rng.choice((0, 0, 8, 5)))
    if op == "edge":
        n, parts = spread(rng, 64, 8192), rng.choice((1, 2, 10))
        T = min(T, 2048 * 2560 * 52 // (n * (4 * parts + 12)))  # bounded by the largest listed case's bytes
        return edge(T, n, parts, rng.choice(("f32", "bf16")), rng.choice(kinds), rng.choice(kinds), rng.random() < 0.7,
                    rng.random() < 0.5, rng.choice(("none", "raw", "sigmoid")), rng.choice((1.0, 0.9)), rng.choice((1.0, 0.5)))
    rank, d_in, d_out = 8 * rng.randint(1, 8), 8 * spread(rng, 8, 320), 8 * spread(rng, 8, 320)
    return adapters(T, spread(rng, 1, min(T, 64)), spread(rng, 1, 32), rank, d_in, d_out, rng.choice(kinds), rng.choice(kinds))


# ------------------------------------------------------------------------------------------------
# Inputs
# ------------------------------------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(seed)
    s = {"case": case}

    def normal(*shape, std=1.0, mean=0.0, type="f32"):
        return (torch.randn(*shape, generator=g, device=dev) * std + mean).to(TYPES[type])

    T = case["T"]
    if case["op"] == "select":
        E, k = case["E"], case["k"]
        l = normal(T, E)
        if T >= MASKED_ROWS:  # some rows find only some of the experts available, one of them none
            rows = torch.arange(0, T, MASKED_ROWS, device=dev)
            l[rows] = torch.where(torch.rand(len(rows), E, generator=g, device=dev) < 0.5, -math.inf, l[rows])
            l[rows[-1]] = -math.inf
        s["logits"] = l.to(TYPES[case["type"]])
        s["bias"] = normal(E, std=0.05) if case["bias"] else None
        s["ids"] = torch.empty(T, k, dtype=torch.int32, device=dev)
        s["weights"] = torch.empty(T, k, device=dev)
    elif case["op"] == "norm":
        n = case["n"]
        s["x"] = normal(T, n + case["pad"], type=case["x"])[:, :n]
        s["gain"] = normal(n, std=0.1, mean=1.0)
        s["out"] = torch.empty(T, n, dtype=TYPES[case["out"]], device=dev)
    elif case["op"] == "edge":
        n, P = case["n"], case["parts"]
        s["parts"] = normal(T, P, n, std=0.5, type=case["part"])
        s["w"] = torch.softmax(normal(T, P), 1) if P > 1 else None
        s["x"] = normal(T, n, type=case["x"])
        s["post_gain"] = normal(n, std=0.1, mean=1.0) if case["post"] else None
        s["channel"] = normal(n, std=0.2, mean=0.8) if case["channel"] else None
        s["token"] = normal(T) if case["token"] != "none" else None
        s["pre_gain"] = normal(n, std=0.1, mean=1.0)
        s["out"] = torch.empty(T, n, dtype=TYPES[case["x"]], device=dev)
        s["next"] = torch.empty(T, n, dtype=TYPES[case["next"]], device=dev)
    else:
        S, n, r, d_in, d_out = case["segments"], case["count"], case["rank"], case["d_in"], case["d_out"]
        host = np.random.RandomState(seed)
        if case["ragged"]:
            cuts = np.sort(host.randint(0, T + 1, S - 1))
            of = host.randint(0, n, S)
            if S >= 8:
                of[host.randint(0, S)] = -1  # a request without an adapter
        else:
            cuts = np.arange(1, S) * T // S
            of = host.permutation(max(S, n))[:S] % n
        s["seg_off"] = torch.tensor(np.concatenate([[0], cuts, [T]]), dtype=torch.int32, device=dev)
        s["seg_adapter"] = torch.tensor(of, dtype=torch.int32, device=dev)
        s["x"] = normal(T, d_in, type=case["x"])
        s["base"] = normal(T, d_out, type=case["y"])
        s["a"] = normal(n, r, d_in, std=d_in ** -0.5, type="bf16")
        s["b"] = normal(n, d_out, r, std=r ** -0.5, type="bf16")
        s["scale"] = torch.rand(n, generator=g, device=dev) * 0.5 + 0.25
        s["y"] = torch.empty(T, d_out, dtype=TYPES[case["y"]], device=dev)
    return s


# ------------------------------------------------------------------------------------------------
# Plain forms
# ------------------------------------------------------------------------------------------------
def plain_select(s, c):
    # scores in 64 bits: which of two near scores is larger must not hang on a rounding
    lowest = torch.finfo(s["logits"].dtype).min
    l = s["logits"].double()
    T, E = l.shape
    masked = torch.isnan(l) | (l <= lowest)
    l = l.clamp(max=F32_MAX).masked_fill(masked, -math.inf)
    if c["score"] == "softmax":
        m = l.amax(1, keepdim=True)
        p = torch.exp(l - torch.where(torch.isinf(m), 0.0, m))
        z = p.sum(1, keepdim=True)
        p = p / torch.where(z == 0, 1.0, z)
    else:
        p = 1.0 / (1.0 + torch.exp(-l))
    value = p if s["bias"] is None else p + s["bias"].double()
    value = value.masked_fill(masked, -math.inf)
    key = l if s["bias"] is None else value
    order = torch.sort(key, dim=1, descending=True, stable=True).indices
    if c["groups"] > 1:
        G = c["groups"]
        best = torch.sort(value.view(T, G, E // G), dim=2, descending=True).values[:, :, :c["group_sum"]]
        none = torch.isinf(best[:, :, 0])
        gs = torch.where(torch.isinf(best), 0.0, best).sum(2).masked_fill(none, -math.inf)
        rank = torch.sort(torch.sort(gs, dim=1, descending=True, stable=True).indices, dim=1).indices
        out = (rank >= c["keep"]).repeat_interleave(E // G, 1)
        late = torch.gather(out, 1, order).to(torch.int32)  # experts of the dropped groups go behind the others
        order = torch.gather(order, 1, torch.sort(late, dim=1, stable=True).indices)
    ids = order[:, :c["k"]]
    w = torch.gather(p, 1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=CLAMP)
    return ids.to(torch.int32), (w * c["scale"]).float()


def rms(v):
    return v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6)


def plain_norm(s, c):
    return (rms(s["x"].float()) * s["gain"]).to(TYPES[c["out"]])


def plain_edge(s, c):
    y = s["parts"].float()
    if s["w"] is not None:
        y = y * s["w"][:, :, None]
    y = y.sum(1)
    if c["post"]:
        y = rms(y) * s["post_gain"]
    if s["channel"] is not None:
        y = y * s["channel"]
    if s["token"] is not None:
        gate = s["token"] if c["token"] == "raw" else 1.0 / (1.0 + torch.exp(-s["token"]))
        y = y * gate[:, None]
    r = c["residual"] * s["x"].float() + c["block"] * y
    return r.to(TYPES[c["x"]]), (rms(r) * s["pre_gain"]).to(TYPES[c["next"]])


def plain_adapters(s, c):
    # every adapter on every token, and the products of a token's own adapter kept
    T, n, r = c["T"], c["count"], c["rank"]
    tokens = torch.arange(T, device=s["x"].device, dtype=torch.int32)
    seg = torch.searchsorted(s["seg_off"], tokens, right=True) - 1
    of = s["seg_adapter"][seg]
    mine = of[:, None] == torch.arange(n, device=of.device)[None, :]
    v = (s["x"].float() @ s["a"].float().reshape(n * r, -1).t()).view(T, n, r) * s["scale"][None, :, None]
    v = torch.where(mine[:, :, None], v, 0.0)
    d = v.view(T, n * r) @ s["b"].float().transpose(1, 2).reshape(n * r, -1)
    return (s["base"].float() + d).to(TYPES[c["y"]])


# ------------------------------------------------------------------------------------------------
# The library's calls
# ------------------------------------------------------------------------------------------------
_ws = {}


def workspace(T):
    """One initialised workspace for each call size, as a serving program keeps them."""
    import quantized_routed_expert_top10_gb300 as qre
    if T not in _ws:
        _ws[T] = torch.empty(qre.strata_moe_workspace_bytes(T), dtype=torch.uint8, device="cuda")
        qre.strata_moe_workspace_init(_ws[T])
    return _ws[T]


def descriptor(s, c, qre):
    """The call's descriptor: a program fills it in once for a layer and keeps it."""
    kind = {"f32": qre.F32, "bf16": qre.BF16, "f16": qre.F16}
    if c["op"] == "select":
        return qre.select(c["E"], c["k"], qre.SCORE_SOFTMAX if c["score"] == "softmax" else qre.SCORE_SIGMOID,
                          n_group=c["groups"], top_group=c["keep"], group_sum=c["group_sum"], renorm=c["renorm"],
                          scale=c["scale"], logits_type=kind[c["type"]])
    if c["op"] == "norm":
        return qre.norm(c["n"], x_type=kind[c["x"]], out_type=kind[c["out"]], x_stride=c["n"] + c["pad"])
    if c["op"] == "edge":
        return qre.combine_norm(c["n"], c["parts"], post_norm=c["post"], token_sigmoid=c["token"] == "sigmoid",
                                residual_scale=c["residual"], block_scale=c["block"], part_type=kind[c["part"]],
                                x_type=kind[c["x"]], next_type=kind[c["next"]])
    return qre.adapters(s["a"], s["b"], c["count"], c["rank"], c["d_in"], c["d_out"], scale=s["scale"], x_type=kind[c["x"]],
                        y_type=kind[c["y"]])


def own_call(s, c):
    import quantized_routed_expert_top10_gb300 as qre
    if "descriptor" not in s:
        s["descriptor"] = descriptor(s, c, qre)
    d, T = s["descriptor"], c["T"]
    if c["op"] == "select":
        qre.strata_moe_select(d, s["logits"], T, s["bias"], s["ids"], s["weights"])
        return s["ids"], s["weights"]
    if c["op"] == "norm":
        qre.strata_moe_norm(d, s["x"], T, s["gain"], s["out"])
        return s["out"]
    if c["op"] == "edge":
        qre.strata_moe_combine_norm(d, s["parts"], s["w"], s["x"], T, s["post_gain"], s["channel"], s["token"], s["pre_gain"],
                                    s["out"], s["next"])
        return s["out"], s["next"]
    qre.strata_moe_adapters(d, s["seg_off"], s["seg_adapter"], c["segments"], s["x"], T, s["base"], s["y"], workspace(T))
    return s["y"]


def run(state):
    c = state["case"]
    if own:
        return own_call(state, c)
    return {"select": plain_select, "norm": plain_norm, "edge": plain_edge, "adapters": plain_adapters}[c["op"]](state, c)


# ------------------------------------------------------------------------------------------------
# What a pass cannot do without
# ------------------------------------------------------------------------------------------------
def work(case):
    c, T = case, case["T"]
    if c["op"] == "select":
        return {"bytes": T * c["E"] * SIZE[c["type"]] + T * c["k"] * 8 + (c["E"] * 4 if c["bias"] else 0), "flops": 8 * T * c["E"]}
    if c["op"] == "norm":
        return {"bytes": T * c["n"] * (SIZE[c["x"]] + SIZE[c["out"]]) + 4 * c["n"], "flops": 4 * T * c["n"]}
    if c["op"] == "edge":
        vectors = 1 + int(c["post"]) + int(c["channel"])
        per = c["parts"] * SIZE[c["part"]] + 2 * SIZE[c["x"]] + SIZE[c["next"]]
        return {"bytes": T * c["n"] * per + 4 * c["n"] * vectors + 4 * T * (c["parts"] if c["parts"] > 1 else 0),
                "flops": T * c["n"] * (2 * c["parts"] + 12)}
    used = min(c["count"], c["segments"], T)
    return {"bytes": T * (c["d_in"] * SIZE[c["x"]] + 2 * c["d_out"] * SIZE[c["y"]]) + 2 * used * c["rank"] * (c["d_in"] + c["d_out"]),
            "flops": 2 * T * c["rank"] * (c["d_in"] + c["d_out"])}


# ------------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ------------------------------------------------------------------------------------------------
def exact_select(s, c):
    T, E, G = c["T"], c["E"], c["groups"]
    lowest = {"f32": np.finfo(np.float32).min, "bf16": float(torch.finfo(torch.bfloat16).min), "f16": -65504.0}[c["type"]]
    logits = s["logits"].float().cpu().numpy().astype(np.float64)
    bias = np.zeros(E) if s["bias"] is None else s["bias"].cpu().numpy().astype(np.float64)
    usable = logits > lowest
    ids, weights = np.zeros((T, c["k"]), np.int32), np.zeros((T, c["k"]))
    for t in range(T):
        l, ok = logits[t], usable[t]
        p = np.zeros(E)
        if ok.any():
            if c["score"] == "softmax":
                e = np.exp(l[ok] - l[ok].max())
                p[ok] = e / math.fsum(e)
            else:
                p[ok] = 1.0 / (1.0 + np.exp(-l[ok]))
        value = p + bias
        groups = range(G)
        if G > 1:
            score = []
            for q in range(G):
                have = np.sort(value[q * (E // G):(q + 1) * (E // G)][ok[q * (E // G):(q + 1) * (E // G)]])[::-1]
                score.append(have[:c["group_sum"]].sum() if len(have) else -math.inf)
            groups = sorted(range(G), key=lambda q: (-score[q], q))[:c["keep"]]
        names = np.concatenate([np.arange(q * (E // G), (q + 1) * (E // G)) for q in sorted(groups)])
        key = np.where(ok, l if s["bias"] is None else value, -math.inf)[names]
        chosen = names[np.lexsort((names, -key))[:c["k"]]]
        w = p[chosen]
        if c["renorm"]:
            w = w / max(w.sum(), CLAMP)
        ids[t], weights[t] = chosen, w * c["scale"]
    return ids, weights


def exact_norm(s, c):
    x = s["x"].double()
    return x / torch.sqrt(x.square().sum(1, keepdim=True) / c["n"] + 1e-6) * s["gain"].double()


def exact_edge(s, c):
    T, n = c["T"], c["n"]
    w = torch.ones(T, c["parts"], dtype=torch.float64, device=s["x"].device) if s["w"] is None else s["w"].double()
    y = torch.einsum("tk,tkn->tn", w, s["parts"].double())
    if c["post"]:
        y = y / torch.sqrt(y.square().sum(1, keepdim=True) / n + 1e-6) * s["post_gain"].double()
    if s["channel"] is not None:
        y = y * s["channel"].double()
    if s["token"] is not None:
        y = y * (s["token"].double() if c["token"] == "raw" else torch.special.expit(s["token"].double()))[:, None]
    r = s["x"].double() * c["residual"] + y * c["block"]
    return r, r / torch.sqrt(r.square().sum(1, keepdim=True) / n + 1e-6) * s["pre_gain"].double()


def exact_adapters(s, c):
    y = s["base"].double()
    off, of = s["seg_off"].tolist(), s["seg_adapter"].tolist()
    for i, a in enumerate(of):
        lo, hi = off[i], off[i + 1]
        if a >= 0 and hi > lo:
            v = s["x"][lo:hi].double() @ s["a"][a].double().t()
            y[lo:hi] += float(s["scale"][a]) * (v @ s["b"][a].double().t())
    return y


def exact(case, seed):
    s = prepare(case, seed)
    return {"select": exact_select, "norm": exact_norm, "edge": exact_edge, "adapters": exact_adapters}[case["op"]](s, case)
