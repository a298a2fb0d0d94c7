"""The operators of strata_moe_ops.h from their definitions, in 64 bits (numpy), and how far fp32 arithmetic may be off.

u = 2^-24 is half a step of fp32.  ``half_step`` is half a step of a result's type, relative to the value."""
import numpy as np
import torch

import quantized_routed_expert_top10_gb300 as qre

TORCH = {qre.F32: torch.float32, qre.BF16: torch.bfloat16, qre.F16: torch.float16}
U = 2.0 ** -24


def half_step(kind):
    return torch.finfo(TORCH[kind]).eps / 2


def to64(t):
    return t.detach().double().cpu().numpy()


# ---- routing -----------------------------------------------------------------------------------------
def select(logits, kind, bias, k, score, n_group=1, top_group=1, group_sum=1, renorm=True, scale=1.0):
    """ids [T][k], weights [T][k] (64 bits) and span [T]: how far below the row's largest logit a chosen one lies."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    lowest = torch.finfo(TORCH[kind]).min
    ids, weights, span = np.zeros((T, k), np.int32), np.zeros((T, k)), np.zeros(T)
    size = E // n_group
    with np.errstate(invalid="ignore"):
        open_ = logits > lowest
        if bias is not None:
            bias = np.asarray(bias, dtype=np.float64)
            open_ &= bias > -np.inf
    for t in range(T):
        l, ok = np.minimum(logits[t], np.finfo(np.float32).max), open_[t]
        p = np.zeros(E)
        if ok.any():
            if score == qre.SCORE_SOFTMAX:
                e = np.exp(l[ok] - l[ok].max())
                p[ok] = e / e.sum()
            else:
                with np.errstate(over="ignore"):
                    p[ok] = 1.0 / (1.0 + np.exp(-l[ok]))
        value = p if bias is None else p + bias
        kept = list(range(n_group))
        if n_group > 1:
            def of_group(g):
                have = sorted((value[e] for e in range(g * size, (g + 1) * size) if ok[e]), reverse=True)
                return sum(have[:group_sum]) if have else -np.inf
            scores = [of_group(g) for g in kept]
            kept = sorted(kept, key=lambda g: (-scores[g], g))[:top_group]
        names = [e for g in sorted(kept) for e in range(g * size, (g + 1) * size)]
        key = {e: (float(l[e]) if bias is None else value[e]) if ok[e] else -np.inf for e in names}
        # a value of -inf is a masked expert's alone, so masked ones come last
        chosen = sorted(names, key=lambda e: (-key[e], e))[:k]
        w = p[chosen]
        if renorm:
            w = w / max(w.sum(), 2.0 ** -14)
        ids[t], weights[t] = chosen, w * np.float64(np.float32(scale))
        if ok.any() and score == qre.SCORE_SOFTMAX:
            span[t] = max([l[ok].max() - l[e] for e in chosen if ok[e]], default=0.0)
    return ids, weights, span


def select_rtol(span):
    """Relative error of a weight in fp32: an exponential of l - m (the difference rounded once: |l - m| u in the
    exponent; the function 4 u), the softmax's sum (positive terms, at most 16 + 5 additions: 21 u), a
    quotient (2 u), the weights' sum (the same errors and at most 32 additions) and a quotient, the scale and the store."""
    return 2 * (np.minimum(span, 104.0) + 4 + 21 + 2) * U + (32 + 4) * U


# ---- norms --------------------------------------------------------------------------------------------
# a mean square of n values: at most 45 additions follow one another in any split over threads and warps (32 values a
# thread, two trees of 5), each 1 u of a sum of positive terms; halved by the root; root, quotient, two products
RMS_U = 45 / 2 + 6


def _row_norm(v):
    return np.sqrt(np.square(v).sum(1, keepdims=True))


def rms_norm(v, v_err, eps, gain):
    """v / sqrt(mean v^2 + eps) * gain of a [T][n] that is off by v_err, and how far fp32 may be off it."""
    n = v.shape[1]
    r = 1.0 / np.sqrt(np.square(v).mean(1, keepdims=True) + np.float64(np.float32(eps)))
    g = 1.0 if gain is None else gain
    out = v * r * g
    # the root's relative change by v_err is at most |v_err| / sqrt(|v|^2 + n eps) as 2-norms
    rel = _row_norm(v_err) / np.sqrt(np.square(v).sum(1, keepdims=True) + n * eps + 1e-300)
    return out, np.abs(r * g) * v_err + np.abs(out) * (RMS_U * U + rel)


def edge(parts, pw, x, post, post_gain, channel, token, sigmoid, pre_gain, eps, residual, block):
    """r, its error, next, its error (before either is rounded to its type); parts [T][P][n] in 64 bits."""
    T, P, n = parts.shape
    w = np.ones((T, P)) if pw is None else pw
    with np.errstate(invalid="ignore"):
        terms = np.where(w[:, :, None] == 0, 0.0, w[:, :, None] * parts)
    y = terms.sum(1)
    y_err = (P + 1) * U * np.abs(terms).sum(1)
    if post:
        y, y_err = rms_norm(y, y_err, eps, post_gain)
    g = np.full((T, 1), np.float64(np.float32(block)))
    if token is not None:
        g = g * ((1.0 / (1.0 + np.exp(-token))) if sigmoid else token)[:, None]
    c = np.ones(n) if channel is None else channel
    gz = g * c * y
    xr = np.float64(np.float32(residual)) * x if x is not None else np.zeros_like(y)
    r = xr + gz
    # the gate: an exponential (4 u), a sum, a quotient, two products; the sum of both: 1 u of each
    r_err = np.abs(g * c) * y_err + 12 * U * np.abs(gz) + 2 * U * np.abs(xr) + U * np.abs(r)
    nx, nx_err = rms_norm(r, r_err, eps, pre_gain)
    return r, r_err, nx, nx_err


def check(got, want, err, kind, what):
    """Every value within its error and its type's rounding (tiny: half a step of the type's smallest numbers)."""
    tiny = {qre.F32: 2.0 ** -149, qre.BF16: 2.0 ** -133, qre.F16: 2.0 ** -24}[kind]
    got = to64(got)
    room = err * (1 + 2 * half_step(kind)) + half_step(kind) * np.abs(want) + tiny
    bad = ~(np.abs(got - want) <= room)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} values off, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} for {want[bad][0]} (room {room[bad][0]:.3g})")


# ---- adapters -------------------------------------------------------------------------------------------
def adapters(x, a, b, scale, seg_off, seg_adapter, base, y0):
    """y [T][d_out] and delta [T][d_out]: rows outside the segments are y0's."""
    y, delta = y0.copy(), np.zeros_like(y0)
    for i, ad in enumerate(seg_adapter):
        lo, hi = seg_off[i], seg_off[i + 1]
        if ad >= 0:
            s = 1.0 if scale is None else scale[ad]
            delta[lo:hi] = s * (x[lo:hi] @ a[ad].T @ b[ad].T)
        y[lo:hi] = delta[lo:hi] + (0.0 if base is None else base[lo:hi])
    return y, delta


def adapters_rtol(d_in, rank, y_kind):
    """2-norm of the error of B (s (A x)) over its own, from the additions that may follow one another in fp32: one for
    every 16 terms of a product and each of up to three bf16 terms of an operand, and 16 for split sums, each off by
    at most a step (the tensor core may cut instead of rounding); and what is left of the inner product
    when it is held as two bf16 terms (16 bits)."""
    adds = 3 * -(-d_in // 16) + 3 * -(-rank // 16) + 16
    return adds * 2 * U + (0.0 if y_kind == qre.F32 else 2.0 ** -16)
