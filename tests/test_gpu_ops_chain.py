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


FIRST_IN_CAPTURE = """
import torch, quantized_routed_expert_top10_gb300 as qre
T, n, E, rank = 2048, 264, 64, 128
x, parts = torch.randn(T, n, device="cuda"), torch.randn(T, 2, n, device="cuda")
odd = torch.randn(T, n + 1, device="cuda")
gain, logits = torch.ones(n, device="cuda"), torch.randn(T, E, device="cuda")
a = torch.randn(2, rank, n, device="cuda").bfloat16()
b = torch.randn(2, n, rank, device="cuda").bfloat16()
off = torch.tensor([0, 1000, T], dtype=torch.int32, device="cuda")
few = torch.tensor([0, 3, 20], dtype=torch.int32, device="cuda")
of = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
ws = torch.empty(qre.strata_moe_workspace_bytes(T), dtype=torch.uint8, device="cuda")
qre.strata_moe_workspace_init(ws)
outs = [torch.zeros(T, n, device="cuda") for _ in range(6)]
odd_out = torch.zeros_like(odd)
ids, w = torch.zeros(T, 4, dtype=torch.int32, device="cuda"), torch.zeros(T, 4, device="cuda")

def calls():
    qre.strata_moe_norm(qre.norm(n), x, T, gain, outs[0])
    qre.strata_moe_norm(qre.norm(n + 1), odd, T, None, odd_out)
    qre.strata_moe_combine_norm(qre.combine_norm(n, 2), parts, None, x, T, gain, None, None, gain, outs[1], outs[2])
    qre.strata_moe_combine_norm(qre.combine_norm(n, 1), outs[1], None, x, T, gain, None, None, None, outs[3], None)
    qre.strata_moe_adapters(qre.adapters(a, b, 2, rank, n, n), off, of, 2, outs[0], T, None, outs[4], ws)
    qre.strata_moe_adapters(qre.adapters(a, b, 2, rank, n, n), few, of, 2, outs[0], T, None, outs[5], ws)
    qre.strata_moe_select(qre.select(E, 4, qre.SCORE_SIGMOID, 8, 4, 2), logits, T, None, ids, w)

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    calls()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (*outs, odd_out, ids, w)]
calls()
torch.cuda.synchronize()
assert qre.strata_poll_status(ws) == 0
assert all(torch.equal(g, t) for g, t in zip(got, (*outs, odd_out, ids, w)))
assert all(g.abs().sum() > 0 for g in got)
"""


def test_first_calls_of_a_process_inside_a_capture():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_IN_CAPTURE], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.parametrize("odd", [0, 1])
def test_rows_further_apart_than_32_bits_count(odd):
    """Rows 2^30 elements and more apart: offsets of elements and bytes beyond 32 bits."""
    T, n, stride = 4, 264 + odd, (1 << 30) + 8
    buf = torch.empty((T - 1) * stride + n, dtype=torch.bfloat16, device=DEV)
    x = torch.as_strided(buf, (T, n), (stride, 1))
    g = torch.Generator(DEV).manual_seed(3)
    x.copy_(torch.randn(T, n, generator=g, device=DEV))
    dense = x.contiguous()
    K16 = qre.BF16

    def same(call):
        """call(rows, stride) for the far rows and for dense ones."""
        far, near = torch.empty(T, n, device=DEV), torch.empty(T, n, device=DEV)
        call(x, stride, far)
        call(dense, n, near)
        torch.cuda.synchronize()
        assert torch.equal(far, near) and (far != 0).any()

    same(lambda v, st, o: qre.strata_moe_norm(qre.norm(n, x_type=K16, x_stride=st), v.data_ptr(), T, None, o))
    same(lambda v, st, o: qre.strata_moe_combine_norm(
        qre.combine_norm(n, 1, x_type=K16, part_type=K16, next_type=qre.F32, part_stride=n, token_stride=st, x_stride=st),
        v.data_ptr(), None, v.data_ptr(), T, None, None, None, None, None, o))
    same(lambda v, st, o: qre.strata_moe_combine_norm(
        qre.combine_norm(n, 4, x_type=K16, part_type=K16, next_type=qre.F32, part_stride=st, token_stride=3 * st + n),
        v.data_ptr(), None, None, 1, None, None, None, None, None, o[0]) or o[1:].zero_())
    # written far apart
    out = torch.empty(T, n, dtype=torch.bfloat16, device=DEV)
    qre.strata_moe_norm(qre.norm(n, x_type=K16, out_type=K16), dense, T, None, out)
    qre.strata_moe_norm(qre.norm(n, x_type=K16, out_type=K16, x_stride=stride, out_stride=stride), x.data_ptr(), T, None, x.data_ptr())
    assert torch.equal(x.contiguous(), out)
    # routing and adapters (dense rows of eights)
    if not odd:
        ids, w, ids2, w2 = (torch.empty(T, 4, dtype=d, device=DEV) for d in (torch.int32, torch.float32) * 2)
        qre.strata_moe_select(qre.select(n, 4, logits_type=K16, logits_stride=stride), x.data_ptr(), T, None, ids, w)
        qre.strata_moe_select(qre.select(n, 4, logits_type=K16), out, T, None, ids2, w2)
        assert torch.equal(ids, ids2) and torch.equal(w, w2)
        a, b = torch.randn(1, 16, n, device=DEV).bfloat16(), torch.randn(1, n, 16, device=DEV).bfloat16()
        off, of = torch.tensor([0, T], dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
        ws = workspace(T)
        near = torch.empty(T, n, device=DEV)
        far = torch.empty(T, n, device=DEV)
        qre.strata_moe_adapters(qre.adapters(a, b, 1, 16, n, n, x_type=K16), off, of, 1, out, T, None, near, ws)
        qre.strata_moe_adapters(qre.adapters(a, b, 1, 16, n, n, x_type=K16, x_stride=stride), off, of, 1, x.data_ptr(), T, None, far, ws)
        assert torch.equal(far, near)
        y = torch.empty(T, n, dtype=torch.bfloat16, device=DEV)
        qre.strata_moe_adapters(qre.adapters(a, b, 1, 16, n, n, y_type=K16), off, of, 1, near, T, out, y, ws)
        qre.strata_moe_adapters(qre.adapters(a, b, 1, 16, n, n, y_type=K16, base_stride=stride, y_stride=stride), off, of, 1, near, T,
                                x.data_ptr(), x.data_ptr(), ws)
        assert torch.equal(x.contiguous(), y)
