"""The hidden values of strata_moe_q4_experts enter the second product with 22 bits whatever the types of x and out: a bf16 result is off by its
own rounding and no more than an fp32 result besides."""
import numpy as np
import pytest
import torch

import ops_reference as ref
import q4_reference as q4ref
import quantized_routed_expert_top10_gb300 as qre
from ops_reference import U

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def half_ulp(v, kind):
    """Half a step of the type at v (normal numbers)."""
    return 2.0 ** np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -100))) * ref.half_step(kind)


def call(gu, dn, x, ids, weights, xk, ok):
    E, T, d_model = gu.count, x.shape[0], x.shape[1]
    p_gu, p_dn = gu.packed(DEV), dn.packed(DEV)
    d = qre.q4_experts(gu.q, p_gu, dn.q, p_dn, E, ids.shape[1], xk, ok)
    ws = torch.empty(qre.strata_moe_q4_experts_workspace_bytes(d, T), dtype=torch.uint8, device=DEV)
    qre.strata_moe_workspace_init(ws)
    out = torch.empty(T, d_model, dtype=ref.TORCH[ok], device=DEV)
    qre.strata_moe_q4_experts(d, torch.from_numpy(ids).to(DEV), torch.from_numpy(weights).to(DEV), x, T, out, ws)
    assert qre.strata_poll_status(ws) == 0
    return ref.to64(out)


@pytest.mark.parametrize("xk", [qre.BF16, qre.F16, qre.F32])
@pytest.mark.parametrize("ok", [qre.BF16, qre.F16])
@pytest.mark.parametrize("T", [4, 64])
def test_single_products(T, xk, ok):
    """x with one column that is not 0 and down with one code a row that is not 8, so that no sum hides a term.  Gate and up are off by 10 u each,
    the hidden value by 2 * 10 + 10 + 8 = 38 u and 4 u for its 22 bits, the output by 8 more: 50 u and half a step of its own type."""
    E, d_model, d_ff = 2, 128, 32
    gu = q4ref.Matrices(E, 2 * d_ff, d_model, 32, paired=True, seed=3)
    dn = q4ref.Matrices(E, d_model, d_ff, 32, seed=4)
    host = np.random.RandomState(3)
    q = np.full((E, d_model, d_ff), 8)
    for e in range(E):
        q[e, np.arange(d_model), host.randint(0, d_ff, d_model)] = host.choice([1, 3, 5, 11, 13, 15], d_model)
    dn.set_codes(q)
    x = torch.zeros(T, d_model)
    x[torch.arange(T), torch.arange(T) * 2] = torch.from_numpy(4.0 + 4.0 * host.random_sample(T)).float()
    x = x.to(ref.TORCH[xk]).to(DEV)
    ids, w = host.randint(0, E, (T, 1)).astype(np.int32), np.ones((T, 1), np.float32)
    got = call(gu, dn, x, ids, w, xk, ok)
    want, _ = q4ref.experts(ref.to64(x), gu, dn, ids, w.astype(np.float64), qre.F32, xk)
    room = half_ulp(want, ok) + 50 * U * np.abs(want)
    if ok == qre.F16:
        room += 2.0 ** -25  # half of fp16's smallest step
    bad = np.abs(got - want) > room
    assert not bad.any(), f"{bad.sum()} of {bad.size} values off by more than their rounding"


@pytest.mark.parametrize("T,E,k,group,zeros", [(1, 12, 3, 32, False), (5, 12, 3, 64, True), (8, 4, 4, 32, False), (64, 256, 4, 32, True), (63, 256, 4, 64, False),
                                               (64, 12, 4, 32, False), (64, 1, 1, 64, False)])
def test_layers(T, E, k, group, zeros):
    """One block and several of an expert's pairs, units of one and two slabs."""
    d_model, d_ff = 192, 448
    gu = q4ref.Matrices(E, 2 * d_ff, d_model, group, zeros, paired=True, seed=5)
    dn = q4ref.Matrices(E, d_model, d_ff, group, zeros, seed=6)
    host = np.random.RandomState(T)
    x = torch.randn(T, d_model, generator=torch.Generator().manual_seed(T)).bfloat16().to(DEV)
    ids = np.argsort(host.random_sample((T, E)), 1)[:, :k].astype(np.int32)
    if E > 100:
        ids[:7, 0], ids[20:45, 1] = 3, 5  # experts of two tiles of columns and of several blocks among many of few pairs
    w = (host.random_sample((T, k)) + 0.05).astype(np.float32)
    got = call(gu, dn, x, ids, w, qre.BF16, qre.BF16)
    want, err = q4ref.experts(ref.to64(x), gu, dn, ids, w.astype(np.float64), qre.F32, qre.BF16)  # the error of an fp32 result
    room = half_ulp(want, qre.BF16) * (1 + 2 * U) + err * (1 + 2 * ref.half_step(qre.BF16))
    bad = np.abs(got - want) > room
    assert not bad.any(), f"{bad.sum()} of {bad.size} values off"
