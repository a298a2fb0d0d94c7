"""The operators as one layer uses them: norm, router logits, request adapters on the logits, routing with groups and a
balance bias, grouping, experts, and the combine with its norms; every step checked on the step's own inputs, and the
whole against the oracle's experts."""
import numpy as np
import pytest
import torch

import gen
import ops_reference as ref
import oracle
import quantized_routed_expert_top10_gb300 as qre
from gpu_common import DEV, BlobCache, check_close, device_packed_layer, to_dev, workspace

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 5, 70])
def test_layer_of_the_separate_operators(T):
    seed, E, n_ad, rank = 31, 512, 3, 16
    g = torch.Generator().manual_seed(T)
    x = to_dev(gen.activations_fast(seed, T))
    gain = (torch.randn(2560, generator=g) * 0.1 + 1).to(DEV)
    post_gain, pre_gain = (torch.randn(2560, generator=g) * 0.1 + 1).to(DEV), (torch.randn(2560, generator=g) * 0.1 + 1).to(DEV)
    token = torch.randn(T, generator=g).to(DEV)
    bias = (torch.randn(E, generator=g) * 0.02).to(DEV)
    wr = to_dev(gen.router_weights(seed, 0))
    a = (torch.randn(n_ad, rank, 2560, generator=g) * 2560 ** -0.5).bfloat16().to(DEV)
    b = (torch.randn(n_ad, E, rank, generator=g) * 0.2).bfloat16().to(DEV)
    cut = T // 3
    off = np.array([0, cut, cut, T], np.int32)
    of = np.array([1, 2, 0], np.int32)
    blobs = device_packed_layer(seed, 0)
    ex = qre.experts(blobs)
    ws = workspace(T)
    empty = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device=DEV)  # noqa: E731
    h, logits, ids10, w10 = empty(T, 2560), empty(T, E), empty(T, 10, dtype=torch.int32), empty(T, 10)
    ids, w, parts = empty(T, 10, dtype=torch.int32), empty(T, 10), empty(T, 10, 2560)
    off_e, pair, active, n_active = (empty(k, dtype=torch.int32) for k in (E + 1, T * 10, E, 1))
    out, nxt = empty(T, 2560), empty(T, 2560)
    adapted = empty(T, E)

    qre.strata_moe_norm(qre.norm(), x, T, gain, h)
    qre.strata_moe_route(h, T, wr, None, E, ids10, w10, logits, ws)
    qre.strata_moe_adapters(qre.adapters(a, b, n_ad, rank, 2560, E), to_dev(off), to_dev(of), 3, h, T, logits, adapted, ws)
    sel = qre.select(E, 10, qre.SCORE_SIGMOID, n_group=8, top_group=4, group_sum=2)
    qre.strata_moe_select(sel, adapted, T, bias, ids, w)
    qre.strata_moe_group(ids, T, E, off_e, pair, active, n_active, ws)
    qre.strata_moe_experts(ex, h, T, off_e, pair, active, n_active, parts, ws)
    qre.strata_moe_combine_norm(qre.combine_norm(token_sigmoid=True, residual_scale=0.9), parts, w, x, T, post_gain, None,
                                token, pre_gain, out, nxt)
    assert qre.strata_poll_status(ws) == 0

    want, err = ref.rms_norm(ref.to64(x), np.zeros((T, 2560)), 1e-6, ref.to64(gain))
    ref.check(h, want, err, qre.F32, "norm")
    want, delta = ref.adapters(ref.to64(h), ref.to64(a), ref.to64(b), None, off, of, ref.to64(logits), np.zeros((T, E)))
    tol = 2 * ref.adapters_rtol(2560, rank, qre.F32) * np.linalg.norm(delta, axis=1) + 2 * ref.U * np.linalg.norm(want, axis=1)
    assert (np.linalg.norm(ref.to64(adapted) - want, axis=1) <= tol).all()
    wid, ww, _ = ref.select(ref.to64(adapted), qre.F32, ref.to64(bias), 10, qre.SCORE_SIGMOID, 8, 4, 2)
    np.testing.assert_array_equal(ids.cpu().numpy(), wid)
    assert np.allclose(ref.to64(w), ww, rtol=float(ref.select_rtol(np.zeros(1))[0]), atol=0)
    # experts: the oracle's parts for the ids chosen
    cache = BlobCache(seed)
    layer = oracle.moe_layer(h.cpu().numpy(), gen.router_weights(seed, 0), None, cache.layer_list(0, wid), q2_offset=1,
                             ids_in=wid, want_parts=True)
    check_close(parts.cpu().numpy().reshape(T, 10, 2560), layer["parts"].reshape(T, 10, 2560), "experts")
    r, r_err, nx, nx_err = ref.edge(ref.to64(parts), ref.to64(w), ref.to64(x), True, ref.to64(post_gain), None,
                                    ref.to64(token), True, ref.to64(pre_gain), 1e-6, 0.9, 1.0)
    ref.check(out, r, r_err, qre.F32, "out")
    ref.check(nxt, nx, nx_err, qre.F32, "next")


def test_chain_in_one_graph_equals_the_calls():
    """Captured once and replayed on new inputs: the same bits as the calls one by one."""
    T, E = 48, 512
    g = torch.Generator().manual_seed(1)
    ws = workspace(T)
    x = torch.randn(T, 2560, generator=g).to(DEV)
    a, b = (torch.randn(2, 8, 2560, generator=g) * 0.02).bfloat16().to(DEV), torch.randn(2, E, 8, generator=g).bfloat16().to(DEV)
    off = torch.tensor([0, 20, 48], dtype=torch.int32, device=DEV)
    of = torch.tensor([1, 0], dtype=torch.int32, device=DEV)
    wr = to_dev(gen.router_weights(2, 0))
    h, logits = torch.empty(T, 2560, device=DEV), torch.empty(T, E, device=DEV)
    ids, w = torch.empty(T, 10, dtype=torch.int32, device=DEV), torch.empty(T, 10, device=DEV)
    parts = torch.randn(T, 10, 2560, generator=g).to(DEV)
    out, nxt = torch.empty(T, 2560, device=DEV), torch.empty(T, 2560, device=DEV)

    def chain():
        qre.strata_moe_norm(qre.norm(), x, T, None, h)
        qre.strata_moe_route(h, T, wr, None, E, ids, w, logits, ws)
        qre.strata_moe_adapters(qre.adapters(a, b, 2, 8, 2560, E), off, of, 2, h, T, logits, logits, ws)
        qre.strata_moe_select(qre.select(E, 10, qre.SCORE_SIGMOID, n_group=16, top_group=4, group_sum=2), logits, T, None, ids, w)
        qre.strata_moe_combine_norm(qre.combine_norm(), parts, w, x, T, None, None, None, None, out, nxt)

    chain()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    x.copy_(torch.randn(T, 2560, generator=g))
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (ids, w, logits, out, nxt)]
    chain()
    assert qre.strata_poll_status(ws) == 0
    for u, v in zip(got, (ids, w, logits, out, nxt)):
        assert torch.equal(u, v)
