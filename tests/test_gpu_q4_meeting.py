"""The meeting of strata_moe_q4_experts' CTAs, run by the wait self-test on a count that nobody else adds to: it runs out within its limit,
reports STRATA_E_TIMEOUT, leaves no copy in flight, and the workspace serves the next call once it is initialised again."""
import time

import numpy as np
import pytest
import torch

import ops_reference as ref
import q4_reference as q4ref
import quantized_routed_expert_top10_gb300 as qre
from gpu_common import workspace

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TIMEOUT = -5


def test_the_meeting_runs_out_as_the_other_waits_do():
    limit = 50_000_000
    ws = workspace(1)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    qre.strata_moe_wait_selftest(ws, limit)
    assert qre.strata_poll_status(ws) == TIMEOUT  # synchronises
    took = time.perf_counter() - t0
    assert 3 * limit * 1e-9 <= took < 1.0  # three waits, one after the other
    # the bit of a meeting that was met after all, or of copies that were not there yet, is not set beside it
    status = ws.view(torch.int32)[:64].cpu()
    assert int(status[0]) == 2
    qre.strata_clear_status(ws)
    assert qre.strata_poll_status(ws) == 0


def test_experts_after_a_meeting_that_ran_out():
    E, k, T, n, d_ff = 6, 2, 5, 128, 64
    gu, dn = q4ref.Matrices(E, 2 * d_ff, n, 32, paired=True), q4ref.Matrices(E, n, d_ff, 32, seed=2)
    p_gu, p_dn = gu.packed(DEV), dn.packed(DEV)
    d = qre.q4_experts(gu.q, p_gu, dn.q, p_dn, E, k)
    host = np.random.RandomState(1)
    ids, w = host.randint(0, E, (T, k)).astype(np.int32), host.random_sample((T, k)).astype(np.float32) + 0.05
    x = torch.randn(T, n, generator=torch.Generator().manual_seed(1)).to(DEV)
    ids_d, w_d, out = torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV), torch.empty(T, n, device=DEV)
    ws = workspace(64)
    assert ws.numel() >= qre.strata_moe_q4_experts_workspace_bytes(d, T)
    for _ in range(2):
        qre.strata_moe_wait_selftest(ws, 20_000)
        assert qre.strata_poll_status(ws) == TIMEOUT
        qre.strata_moe_workspace_init(ws)
        out.zero_()
        qre.strata_moe_q4_experts(d, ids_d, w_d, x, T, out, ws)
        assert qre.strata_poll_status(ws) == 0
        want, err = q4ref.experts(ref.to64(x), gu, dn, ids, w.astype(np.float64), qre.F32)
        ref.check(out, want, err, qre.F32, "after a timeout")
