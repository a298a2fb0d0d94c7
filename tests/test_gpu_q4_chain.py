"""A routed-expert layer of any shape put together from the library's calls: norm, router, routing, experts with 4-bit weights, a projection, and
the norm of the next layer; call by call against the formulas, and as a captured graph that is replayed with other inputs."""
import numpy as np
import pytest
import torch

import ops_reference as ref
import q4_reference as q4ref
import quantized_routed_expert_top10_gb300 as qre

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("T", [1, 4, 33])
def test_layer_call_by_call_and_as_a_graph(T):
    E, k, n, d_ff, shared = 24, 4, 384, 160, 24
    g = torch.Generator().manual_seed(T)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, gain, pre_gain = rnd(T, n).to(DEV), (1 + 0.1 * rnd(n)).to(DEV), (1 + 0.1 * rnd(n)).to(DEV)
    router = (rnd(E, n) * n ** -0.5).bfloat16().to(DEV)
    bias, balance = (0.1 * rnd(E)).to(DEV), (0.02 * rnd(E)).to(DEV)
    gu = q4ref.Matrices(E + 1, 2 * d_ff, n, 32, True, paired=True, seed=5)  # the last one: a shared expert that every token lists
    dn = q4ref.Matrices(E + 1, n, d_ff, 32, True, seed=6)
    proj = q4ref.Matrices(1, 200, n, 64, seed=7)
    p_gu, p_dn, p_proj = gu.packed(DEV), dn.packed(DEV), proj.packed(DEV)
    ex = qre.q4_experts(gu.q, p_gu, dn.q, p_dn, E + 1, k + 1)
    ws = torch.zeros(qre.strata_moe_q4_experts_workspace_bytes(ex, T), dtype=torch.uint8, device=DEV)
    qre.strata_moe_workspace_init(ws)
    empty = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device=DEV)  # noqa: E731
    h, logits, ids, w = empty(T, n), empty(T, E), empty(T, k, dtype=torch.int32), empty(T, k)
    ids1 = torch.full((T, k + 1), shared, dtype=torch.int32, device=DEV)
    w1 = torch.ones(T, k + 1, device=DEV)
    moe, out, nxt, y = empty(T, n), empty(T, n), empty(T, n), empty(T, 200)
    sel = qre.select(E, k, qre.SCORE_SIGMOID, n_group=4, top_group=2, group_sum=2)
    lin, head = qre.linear_bf16(router, E, n), qre.linear_q4(proj.q, p_proj)
    cn = qre.combine_norm(n, 1, post_norm=False)

    def layer():
        qre.strata_moe_norm(qre.norm(n), x, T, gain, h)
        qre.strata_moe_linear(lin, h, T, bias, logits)
        qre.strata_moe_select(sel, logits, T, balance, ids, w)
        ids1[:, :k].copy_(ids)
        w1[:, :k].copy_(w)
        qre.strata_moe_q4_experts(ex, ids1, w1, h, T, moe, ws)
        qre.strata_moe_combine_norm(cn, moe, None, x, T, None, None, None, pre_gain, out, nxt)
        qre.strata_moe_linear(head, nxt, T, None, y)

    def check():
        assert qre.strata_poll_status(ws) == 0
        h64 = ref.to64(h)
        want, err = ref.rms_norm(ref.to64(x), np.zeros((T, n)), 1e-6, ref.to64(gain))
        ref.check(h, want, err, qre.F32, "norm")
        want, err = q4ref.product(h64, np.zeros_like(h64), ref.to64(router), q4ref.additions(n, 128))
        want = want + ref.to64(bias)
        ref.check(logits, want, err + ref.U * np.abs(want), qre.F32, "router")
        wid, ww, _ = ref.select(ref.to64(logits), qre.F32, ref.to64(balance), k, qre.SCORE_SIGMOID, 4, 2, 2)
        np.testing.assert_array_equal(ids.cpu().numpy(), wid)
        assert np.allclose(ref.to64(w), ww, rtol=float(ref.select_rtol(np.zeros(1))[0]), atol=0)
        want, err = q4ref.experts(h64, gu, dn, ids1.cpu().numpy(), ref.to64(w1), qre.F32)
        ref.check(moe, want, err, qre.F32, "experts")
        r, r_err, nx, nx_err = ref.edge(ref.to64(moe)[:, None], None, ref.to64(x), False, None, None, None, False, ref.to64(pre_gain), 1e-6, 1.0,
                                        1.0)
        ref.check(out, r, r_err, qre.F32, "residual")
        ref.check(nxt, nx, nx_err, qre.F32, "next norm")
        n64 = ref.to64(nxt)
        want, err = q4ref.product(n64, q4ref.held(n64, 22), proj.weights(0), q4ref.additions(n, 64))
        ref.check(y, want, err, qre.F32, "projection")

    layer()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    for seed in (11, 12, 13):
        x.copy_(torch.randn(T, n, generator=torch.Generator().manual_seed(seed)))
        y.zero_()
        graph.replay()
        check()
