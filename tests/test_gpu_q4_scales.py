"""Scales far from 1 beside activations far from 1: the largest that strata_moe_ops.h allows, the smallest of their types, results of ordinary size."""
import numpy as np
import pytest
import torch

import ops_reference as ref
import q4_reference as q4ref
import quantized_routed_expert_top10_gb300 as qre

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("kind,scale,size", [(qre.BF16, 2.0 ** 99, 2.0 ** -95), (qre.BF16, 2.0 ** -120, 2.0 ** 110), (qre.BF16, 2.0 ** -133, 2.0 ** 120),
                                             (qre.F16, 65504.0, 2.0 ** -60), (qre.F16, 2.0 ** -24, 2.0 ** 60), (qre.BF16, 2.0 ** 99, 2.0 ** -126)])
@pytest.mark.parametrize("T,group", [(1, 32), (5, 64), (30, 128)])
def test_scales_far_from_one(kind, scale, size, T, group):
    d_in, n_out = 640 + group, 72
    m = q4ref.Matrices(1, n_out, d_in, group, zeros=True, scale_type=kind)
    sign = torch.where(torch.rand(m.scales.shape, generator=torch.Generator().manual_seed(2)) < 0.5, -1.0, 1.0)
    m.scales = (sign * scale).to(ref.TORCH[kind])
    assert torch.isfinite(m.scales).all() and (m.scales != 0).all()
    packed = m.packed(DEV)
    x = (torch.randn(T, d_in, generator=torch.Generator().manual_seed(3)) * size).to(DEV)
    y = torch.empty(T, n_out, device=DEV)
    qre.strata_moe_linear(qre.linear_q4(m.q, packed), x, T, None, y)
    x64 = ref.to64(x)
    want, err = q4ref.product(x64, q4ref.held(x64, 22), m.weights(0), q4ref.additions(d_in, group))
    assert np.abs(want).max() < 2.0 ** 120
    ref.check(y, want, err + 2.0 ** -149 * q4ref.additions(d_in, group), qre.F32, f"scales of {scale}")
