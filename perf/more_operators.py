"""Products of a few tokens with 4-bit weights: what is timed, their plain forms and their exact values.

  linear    strata_moe_linear: one projection of a few tokens, by 4-bit weights with group scales or, as routers
            have them, by bf16 weights
  experts   strata_moe_q4_experts: the routed experts of a few tokens (gate, up, SwiGLU, down and the weighted sum)
            with 4-bit weights, after routing

A 4-bit weight is scale * (code - zero): codes 0..15, two to a byte (the even column in the low bits), a scale for
each row and group of columns, and a zero point for each of them or 8.  The plain forms are elementary torch
operations; with ``own`` set, run() makes the library's calls.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------------------------------------
# Cases
# ------------------------------------------------------------------------------------------------
def linear(T, d_in, n_out, weight, x, y, group=64, zeros=False, scale="bf16", bias=False, **name):
    return dict(name, op="linear", T=T, d_in=d_in, n_out=n_out, weight=weight, x=x, y=y, group=group, zeros=zeros, scale=scale,
                bias=bias)


def experts(T, E, k, d_model, d_ff, x, out, group=64, zeros=False, scale="bf16", window=False, shared=False, drop=False, **name):
    return dict(name, op="experts", T=T, E=E, k=k, d_model=d_model, d_ff=d_ff, x=x, out=out, group=group, zeros=zeros,
                scale=scale, window=window, shared=shared, drop=drop)


def listed():
    return [
        # one decoded token through a projection beside the block, from the model's width to itself
        linear(1, 2560, 2560, "q4", "f32", "f32", group=64, name="linear decode"),
        # a verify window of four through a wide projection, zero points, bf16 activations
        linear(4, 2560, 10240, "q4", "bf16", "bf16", group=128, zeros=True, name="linear verify"),
        # one token's logits over a vocabulary
        linear(1, 2560, 131072, "q4", "bf16", "f32", group=32, name="linear vocabulary"),
        # 64 requests decoding together
        linear(64, 2560, 10240, "q4", "bf16", "bf16", group=32, bias=True, name="linear batch"),
        # a ragged batch and an odd number of rows, fp16 activations and scales
        linear(13, 1184, 2051, "q4", "f16", "f16", group=32, zeros=True, scale="f16", bias=True, name="linear ragged f16"),
        # the router's logits of one token
        linear(1, 2560, 512, "bf16", "f32", "f32", name="router decode"),
        # the router's logits of 64 requests
        linear(64, 2560, 512, "bf16", "f32", "f32", bias=True, name="router batch"),
        # one token's ten experts of 512, the layer's own sizes
        experts(1, 512, 10, 2560, 640, "f32", "f32", name="experts decode"),
        # a verify window of four related tokens
        experts(4, 512, 10, 2560, 640, "f32", "f32", window=True, name="experts verify"),
        # 64 requests decoding together: most of the experts, one or two tokens each
        experts(64, 512, 10, 2560, 640, "bf16", "bf16", group=32, name="experts batch"),
        # 16 requests of a layer of fewer and larger experts, zero points, fp16
        experts(16, 64, 6, 2048, 1024, "f16", "f16", group=128, zeros=True, scale="f16", name="experts few f16"),
        # a small layer of odd sizes: a shared expert as the last of each token's list, slots without an expert
        experts(7, 60, 5, 1184, 416, "bf16", "f32", group=32, zeros=True, shared=True, drop=True, name="experts ragged"),
    ]


def spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kinds = ("f32", "bf16", "f16")
    T, group = spread(rng, 1, 64), rng.choice((32, 64, 128))
    x, y = rng.choice(kinds), rng.choice(kinds)
    zeros, scale = rng.random() < 0.5, rng.choice(("bf16", "bf16", "f16"))
    if rng.random() < 0.5:
        if rng.random() < 0.25:
            return linear(T, 8 * spread(rng, 8, 512), spread(rng, 8, 1024), "bf16", x, y, bias=rng.random() < 0.5)
        d_in = group * spread(rng, max(1, 64 // group), 8192 // group)
        return linear(T, d_in, min(spread(rng, 16, 32768), 64 * 2560 * 10240 // (T * d_in)), "q4", x, y, group, zeros, scale,
                      rng.random() < 0.5)
    d_model = group * spread(rng, max(1, 128 // group), 4096 // group)
    d_ff = group * spread(rng, max(1, 128 // group), 2048 // group)
    d_ff = max(group, min(d_ff, 2560 * 1024 // d_model // group * group))
    E = min(spread(rng, 4, 512), 512 * 2560 * 640 // (d_model * d_ff))
    k = rng.randint(1, min(10, E - 1))
    T = max(1, min(T, 640 * 2560 * 640 // (k * d_model * d_ff)))
    return experts(T, E, k, d_model, d_ff, x, y, group, zeros, scale, rng.random() < 0.3, rng.random() < 0.3, rng.random() < 0.3)


# ------------------------------------------------------------------------------------------------
# Inputs
# ------------------------------------------------------------------------------------------------
def routing(c, seed):
    """ids int32 [T][k] and weights fp32 [T][k]: the k largest of random logits and their softmax."""
    host = np.random.RandomState(seed)
    T, E, k = c["T"], c["E"], c["k"]
    logits = host.standard_normal((T, E))
    if c["window"]:  # tokens that follow one another choose alike
        logits = logits[:1] + 0.3 * logits
    if c["shared"]:  # the last expert takes every token, with weight 1
        logits[:, E - 1] = -np.inf
    routed = k - 1 if c["shared"] and k > 1 else k
    ids = np.argsort(-logits, axis=1)[:, :routed]
    w = np.exp(np.take_along_axis(logits, ids, 1))
    w = w / w.sum(1, keepdims=True)
    if routed < k:
        ids = np.concatenate([ids, np.full((T, 1), E - 1)], 1)
        w = np.concatenate([w, np.ones((T, 1))], 1)
    if c["drop"]:  # slots without an expert, and a token without any weight
        gone = host.random_sample((T, k)) < 0.1
        w[gone] = 0.0
        ids[gone] = -1
        if T >= 4:
            w[host.randint(0, T)] = 0.0
    return ids.astype(np.int32), w.astype(np.float32)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(seed)
    c = case
    s = {"case": case}

    def normal(*shape, std=1.0, type="f32"):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(TYPES[type])

    def matrices(count, n_out, d_in):
        """count 4-bit matrices whose products with x ~ N(0, 1) are about as large as x."""
        groups = d_in // c["group"]
        m = {"codes": torch.randint(0, 256, (count, n_out, d_in // 2), dtype=torch.uint8, generator=g, device=dev)}
        m["scales"] = ((torch.rand(count, n_out, groups, generator=g, device=dev) + 0.5) * (d_in ** -0.5 / 4.6)).to(TYPES[c["scale"]])
        m["zeros"] = None
        if c["zeros"]:
            m["zeros"] = torch.randint(5, 11, (count, n_out, groups), dtype=torch.uint8, generator=g, device=dev)
        return m

    T = c["T"]
    if c["op"] == "linear":
        s["x"] = normal(T, c["d_in"], type=c["x"])
        if c["weight"] == "q4":
            s["w"] = matrices(1, c["n_out"], c["d_in"])
        else:
            s["w"] = normal(c["n_out"], c["d_in"], std=c["d_in"] ** -0.5, type="bf16")
        s["bias"] = normal(c["n_out"], std=0.1) if c["bias"] else None
        s["y"] = torch.empty(T, c["n_out"], dtype=TYPES[c["y"]], device=dev)
    else:
        s["x"] = normal(T, c["d_model"], type=c["x"])
        s["gate_up"] = matrices(c["E"], 2 * c["d_ff"], c["d_model"])  # rows of gate, then rows of up
        s["down"] = matrices(c["E"], c["d_model"], c["d_ff"])
        ids, w = routing(c, seed)
        s["ids"], s["weights"] = torch.from_numpy(ids).to(dev), torch.from_numpy(w).to(dev)
        s["out"] = torch.empty(T, c["d_model"], dtype=TYPES[c["out"]], device=dev)
    if own:
        plan(s, c)
    return s


# ------------------------------------------------------------------------------------------------
# Plain forms
# ------------------------------------------------------------------------------------------------
def widen(codes, scales, zeros, group):
    """fp32 weights [..., rows, columns] of 4-bit codes."""
    q = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).float()
    q = q.unflatten(-1, (-1, group))
    z = 8.0 if zeros is None else zeros.float().unsqueeze(-1)
    return ((q - z) * scales.float().unsqueeze(-1)).flatten(-2)


def plain_linear(s, c):
    if c["weight"] == "q4":
        w = widen(s["w"]["codes"][0], s["w"]["scales"][0], None if s["w"]["zeros"] is None else s["w"]["zeros"][0], c["group"])
    else:
        w = s["w"].float()
    y = s["x"].float() @ w.t()
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(TYPES[c["y"]])


def plain_experts(s, c):
    def of(m, e):
        """The weights of expert e[t] for each token."""
        return widen(m["codes"][e], m["scales"][e], None if m["zeros"] is None else m["zeros"][e], c["group"])

    x = s["x"].float().unsqueeze(2)
    y = torch.zeros(c["T"], c["d_model"], device=x.device)
    for i in range(c["k"]):
        e = s["ids"][:, i].clamp(min=0).long()
        gu = (of(s["gate_up"], e) @ x).squeeze(2)
        gate, up = gu[:, :c["d_ff"]], gu[:, c["d_ff"]:]
        h = gate / (1.0 + torch.exp(-gate)) * up
        part = (of(s["down"], e) @ h.unsqueeze(2)).squeeze(2)
        w = torch.where(s["ids"][:, i] >= 0, s["weights"][:, i], 0.0)
        y = y + w[:, None] * part
    return y.to(TYPES[c["out"]])


# ------------------------------------------------------------------------------------------------
# The library's calls
# ------------------------------------------------------------------------------------------------
def plan(s, c):
    """What a serving program makes once for a layer: packed weights, the descriptor, a workspace."""
    import quantized_routed_expert_top10_gb300 as qre
    kind = {"f32": qre.F32, "bf16": qre.BF16, "f16": qre.F16}

    def packed(m, paired):
        count, n_out, half = m["codes"].shape
        q = qre.q4(n_out, 2 * half, c["group"], zeros=c["zeros"], scale_type=kind[c["scale"]], paired=paired)
        to = torch.empty(count, qre.strata_q4_bytes(q), dtype=torch.uint8, device=m["codes"].device)
        qre.strata_pack_q4_device(q, m["codes"], m["scales"], m["zeros"], to, count)
        return q, to

    if c["op"] == "linear":
        if c["weight"] == "q4":
            q, s["packed"] = packed(s["w"], False)
            s["descriptor"] = qre.linear_q4(q, s["packed"], x_type=kind[c["x"]], y_type=kind[c["y"]])
        else:
            s["descriptor"] = qre.linear_bf16(s["w"], c["n_out"], c["d_in"], x_type=kind[c["x"]], y_type=kind[c["y"]])
        return
    qg, s["packed_gate_up"] = packed(s["gate_up"], True)
    qd, s["packed_down"] = packed(s["down"], False)
    s["descriptor"] = qre.q4_experts(qg, s["packed_gate_up"], qd, s["packed_down"], c["E"], c["k"], x_type=kind[c["x"]],
                                     out_type=kind[c["out"]])
    s["ws"] = torch.empty(qre.strata_moe_q4_experts_workspace_bytes(s["descriptor"], c["T"]), dtype=torch.uint8, device="cuda")
    qre.strata_moe_workspace_init(s["ws"])


def own_call(s, c):
    import quantized_routed_expert_top10_gb300 as qre
    if "descriptor" not in s:
        plan(s, c)
    if c["op"] == "linear":
        qre.strata_moe_linear(s["descriptor"], s["x"], c["T"], s["bias"], s["y"])
        return s["y"]
    qre.strata_moe_q4_experts(s["descriptor"], s["ids"], s["weights"], s["x"], c["T"], s["out"], s["ws"])
    return s["out"]


def run(state):
    c = state["case"]
    if own:
        return own_call(state, c)
    return plain_linear(state, c) if c["op"] == "linear" else plain_experts(state, c)


# ------------------------------------------------------------------------------------------------
# What a pass cannot do without
# ------------------------------------------------------------------------------------------------
def matrix_bytes(c, n_out, d_in):
    return n_out * (d_in // 2 + d_in // c["group"] * (3 if c["zeros"] else 2))


def work(case):
    c, T = case, case["T"]
    if c["op"] == "linear":
        weights = 2 * c["n_out"] * c["d_in"] if c["weight"] == "bf16" else matrix_bytes(c, c["n_out"], c["d_in"])
        return {"bytes": weights + T * (c["d_in"] * SIZE[c["x"]] + c["n_out"] * SIZE[c["y"]]) + (4 * c["n_out"] if c["bias"] else 0),
                "flops": 2 * T * c["n_out"] * c["d_in"]}
    used = pairs = 0.0
    for seed in range(4):  # experts that some token weighs, on average
        ids, w = routing(c, seed)
        used += len(np.unique(ids[w != 0])) / 4
        pairs += np.count_nonzero(w) / 4
    one = matrix_bytes(c, 2 * c["d_ff"], c["d_model"]) + matrix_bytes(c, c["d_model"], c["d_ff"])
    return {"bytes": used * one + T * (c["d_model"] * (SIZE[c["x"]] + SIZE[c["out"]]) + 8 * c["k"]),
            "flops": 6 * pairs * c["d_model"] * c["d_ff"]}


# ------------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ------------------------------------------------------------------------------------------------
def exact_product(x, m, i, group):
    """x [T][columns] by matrix i: for each group scale * (sum of code * x - zero * sum of x)."""
    T, columns = x.shape
    n = columns // group
    xg = x.view(T, n, group)
    out = torch.empty(T, m["codes"].shape[1], dtype=torch.float64, device=x.device)
    for lo in range(0, out.shape[1], 8192):
        b = m["codes"][i, lo:lo + 8192]
        rows = b.shape[0]
        q = torch.empty(rows, columns, dtype=torch.float64, device=x.device)
        q[:, 0::2] = b.remainder(16)
        q[:, 1::2] = b.div(16, rounding_mode="floor")
        part = torch.einsum("rgi,tgi->trg", q.view(rows, n, group), xg)
        zero = torch.full((rows, n), 8.0, dtype=torch.float64, device=x.device)
        if m["zeros"] is not None:
            zero = m["zeros"][i, lo:lo + 8192].double()
        part = part - zero[None] * xg.sum(2)[:, None, :]
        out[:, lo:lo + 8192] = (part * m["scales"][i, lo:lo + 8192].double()[None]).sum(2)
    return out


def exact_linear(s, c):
    x = s["x"].double()
    y = exact_product(x, s["w"], 0, c["group"]) if c["weight"] == "q4" else torch.einsum("tk,nk->tn", x, s["w"].double())
    return y if s["bias"] is None else y + s["bias"].double()[None]


def exact_experts(s, c):
    x, F = s["x"].double(), c["d_ff"]
    y = torch.zeros(c["T"], c["d_model"], dtype=torch.float64, device=x.device)
    ids, w = s["ids"].cpu().numpy(), s["weights"].cpu().numpy().astype(np.float64)
    for e in np.unique(ids[ids >= 0]):
        t, i = np.nonzero(ids == e)
        rows = torch.from_numpy(t).to(x.device)
        gu = exact_product(x[rows], s["gate_up"], int(e), c["group"])
        h = gu[:, :F] * torch.special.expit(gu[:, :F]) * gu[:, F:]
        part = exact_product(h, s["down"], int(e), c["group"])
        y.index_add_(0, rows, part * torch.from_numpy(w[t, i]).to(x.device)[:, None])
    return y


def exact(case, seed):
    s = prepare(case, seed)
    return exact_linear(s, case) if case["op"] == "linear" else exact_experts(s, case)
