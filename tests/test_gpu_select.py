"""strata_moe_select against its definition in 64 bits: ids exactly, weights to fp32's rounding."""
import numpy as np
import pytest
import torch

import ops_reference as ref
import quantized_routed_expert_top10_gb300 as qre

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SOFT, SIG = qre.SCORE_SOFTMAX, qre.SCORE_SIGMOID


def run(logits, kind, bias, k, score, **kw):
    """ids, weights of a call; logits: CPU float tensor [T][stride] of which the first E columns count."""
    E = kw.pop("E", logits.shape[1])
    l = logits.to(ref.TORCH[kind]).to(DEV)
    T = l.shape[0]
    ids = torch.full((T + 1, k), -7, dtype=torch.int32, device=DEV)
    w = torch.full((T + 1, k), -7.0, device=DEV)
    b = None if bias is None else bias.to(DEV)
    sel = qre.select(E, k, score, logits_type=kind, logits_stride=l.shape[1], **kw)
    qre.strata_moe_select(sel, l, T, b, ids, w)
    torch.cuda.synchronize()
    assert (ids[T] == -7).all() and (w[T] == -7).all()  # nothing past the last token
    want, ww, span = ref.select(ref.to64(l[:, :E]), kind, None if bias is None else ref.to64(bias), k, score, **kw)
    got, gw = ids[:T].cpu().numpy(), ref.to64(w[:T])
    np.testing.assert_array_equal(got, want)
    room = np.abs(ww) * ref.select_rtol(span)[:, None] + 2.0 ** -126
    assert (np.abs(gw - ww) <= room).all(), np.max(np.abs(gw - ww) / room)
    return got, gw


def randn(*shape, seed=0, std=1.0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std


GROUPS = {1: (1, 1, 1), 4: (4, 2, 1), 8: (8, 3, 2), 16: (16, 4, 2), 32: (32, 32, 1)}


@pytest.mark.parametrize("kind", [qre.F32, qre.BF16, qre.F16])
@pytest.mark.parametrize("score", [SOFT, SIG])
@pytest.mark.parametrize("T,E,k,groups,bias,renorm", [
    (1, 512, 10, 1, False, True), (300, 512, 10, 16, True, True), (129, 160, 6, 8, False, False),
    (64, 32, 10, 1, True, True), (33, 1, 1, 1, True, True), (7, 31, 31, 1, False, True), (50, 96, 32, 32, True, False),
    (65, 500, 12, 4, True, True), (40, 7, 3, 1, True, False), (1001, 512, 1, 16, False, True)])
def test_against_definition(kind, score, T, E, k, groups, bias, renorm):
    G, keep, gsum = GROUPS[groups]
    run(randn(T, E, seed=T + E), kind, randn(E, seed=5, std=0.1) if bias else None, k, score, n_group=G, top_group=keep,
        group_sum=gsum, renorm=renorm, scale=2.5 if bias else 1.0)


def test_largest_call_and_strided_rows():
    run(randn(8192, 520, seed=1), qre.F32, randn(512, seed=2, std=0.05), 10, SIG, E=512, n_group=16, top_group=4, group_sum=2,
        scale=2.5)
    run(randn(257, 517, seed=3), qre.BF16, None, 8, SOFT, E=511)


@pytest.mark.parametrize("score", [SOFT, SIG])
@pytest.mark.parametrize("bias", [False, True])
def test_ties_go_to_the_lower_id(score, bias):
    # few distinct logits: mass ties inside the top k and around its end, groups of equal scores
    T, E = 96, 512
    l = torch.randint(-2, 3, (T, E), generator=torch.Generator().manual_seed(4)).float()
    l[0] = 0.0
    l[1] = -0.0
    l[2, ::2] = -0.0
    b = torch.zeros(E) if bias else None
    for groups in (1, 8, 16):
        G, keep, gsum = GROUPS[groups]
        ids, _ = run(l, qre.F32, b, 10, score, n_group=G, top_group=keep, group_sum=gsum)
        if groups == 1:
            assert ids[0].tolist() == list(range(10)) and ids[1].tolist() == list(range(10))


@pytest.mark.parametrize("score", [SOFT, SIG])
@pytest.mark.parametrize("kind", [qre.F32, qre.BF16, qre.F16])
def test_masked_experts(score, kind):
    T, E = 64, 128
    lowest = torch.finfo(ref.TORCH[kind]).min
    l = randn(T, E, seed=6)
    for t, mask in enumerate((-np.inf, lowest, float("nan"))):
        l[t] = mask                                        # nothing is left
        l[3 + t, 1:] = mask                                # one expert is left, fewer than k
        l[6 + t, : E // 2] = mask                          # half the groups are empty
        l[9 + t, torch.arange(E) % 16 >= 3] = mask         # three in each group
    l[12, 5] = float("nan")
    l[13, 7] = np.inf                                      # +inf: the largest finite value
    l[14, 3:9] = np.inf
    for bias in (None, randn(E, seed=7, std=0.3)):
        if bias is not None:
            bias[3] = -np.inf
            bias[9] = float("nan")
        for groups in (1, 8):
            G, keep, gsum = GROUPS[groups]
            for renorm in (True, False):
                ids, w = run(l, kind, bias, 10, score, n_group=G, top_group=keep, group_sum=gsum, renorm=renorm)
                assert (w[:3] == 0).all() and np.isfinite(w).all()
                assert all(len(set(r)) == 10 for r in ids.tolist()) and ids.min() >= 0 and ids.max() < E


def test_bias_of_infinity_forces_an_expert():
    b = torch.zeros(64)
    b[[40, 50]] = np.inf
    ids, _ = run(randn(20, 64, seed=8), qre.F32, b, 4, SIG)
    assert (ids[:, 0] == 40).all() and (ids[:, 1] == 50).all()
    run(randn(20, 64, seed=8), qre.F32, b, 4, SIG, n_group=8, top_group=2, group_sum=2)


def test_values_that_32_bits_cannot_tell_apart():
    """Pairs of experts whose value differs by far less than a step of fp32, in either order of their ids."""
    T, E = 200, 64
    g = np.random.default_rng(9)
    l = np.full((T, E), -4.0, np.float32) + g.uniform(-0.1, 0.1, (T, E)).astype(np.float32)
    b = g.uniform(-0.01, 0.01, E).astype(np.float32)
    for t in range(T):
        e = g.choice(E, 6, replace=False)
        for i in range(0, 6, 2):
            # sigmoid(l0) + b0 ~ sigmoid(l1) + b1: l1 found in 64 bits, then rounded to fp32
            l[t, e[i]] = g.uniform(0.5, 2.0)
            v = 1 / (1 + np.exp(-np.float64(l[t, e[i]]))) + np.float64(b[e[i]]) - np.float64(b[e[i + 1]])
            l[t, e[i + 1]] = np.float32(np.log(v / (1 - v)))
    lt, bt = torch.from_numpy(l), torch.from_numpy(b)
    for k in (1, 2, 3, 6, 7):
        run(lt, qre.F32, bt, k, SIG)
    run(lt, qre.F32, bt, 5, SIG, n_group=8, top_group=4, group_sum=2)
    run(lt, qre.F32, bt, 5, SIG, n_group=8, top_group=1, group_sum=1)
    # the same under a softmax: p0 + b0 ~ p1 + b1 with biases made to fit p
    for t in range(0, T, 10):
        row = lt[t:t + 1].double().numpy()[0]
        p = np.exp(row - row.max())
        p /= p.sum()
        order = np.argsort(-p)
        bb = np.zeros(E)
        bb[order[1]] = p[order[0]] - p[order[1]]
        bb[order[3]] = p[order[2]] - p[order[3]]
        bb = torch.from_numpy(bb.astype(np.float32))
        run(lt[t:t + 1], qre.F32, bb, 4, SOFT)
        run(lt[t:t + 1], qre.F32, bb, 4, SOFT, n_group=4, top_group=2, group_sum=2)


def test_far_logits():
    # scores that saturate (sigmoid: many round to 1) or vanish (softmax): the order is the logits'
    l = randn(40, 256, seed=10, std=60.0)
    for score in (SOFT, SIG):
        for renorm in (True, False):
            run(l, qre.F32, None, 10, score, renorm=renorm)
        run(l, qre.F32, None, 10, score, n_group=8, top_group=4, group_sum=1)
    run(randn(40, 256, seed=11, std=1e-6), qre.F32, None, 10, SOFT)
    run(randn(40, 256, seed=12, std=1e-6), qre.F32, randn(256, seed=13, std=1e-6), 10, SIG)
    # weights whose sum is below the clamp
    run(randn(40, 256, seed=14) - 30.0, qre.F32, None, 10, SIG)


def test_repeats_streams_and_graphs():
    T, E, k = 500, 512, 10
    l, b = randn(T, E, seed=15).to(DEV), randn(E, seed=16, std=0.1).to(DEV)
    sel = qre.select(E, k, SIG, n_group=16, top_group=4, group_sum=2)
    ids, w = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
    qre.strata_moe_select(sel, l, T, b, ids, w)
    torch.cuda.synchronize()
    first = ids.clone(), w.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ids.zero_(), w.zero_()
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        qre.strata_moe_select(sel, l, T, b, ids, w)
    side.synchronize()
    assert torch.equal(ids, first[0]) and torch.equal(w, first[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qre.strata_moe_select(sel, l, T, b, ids, w)
    l.copy_(randn(T, E, seed=17))
    graph.replay()
    torch.cuda.synchronize()
    want, _, _ = ref.select(ref.to64(l), qre.F32, ref.to64(b), k, SIG, 16, 4, 2)
    np.testing.assert_array_equal(ids.cpu().numpy(), want)


@pytest.mark.parametrize("score", [SOFT, SIG])
@pytest.mark.parametrize("kind", [qre.F32, qre.BF16, qre.F16])
def test_bias_of_infinity_brings_no_masked_expert_back(score, kind):
    T, E = 48, 64
    l = randn(T, E, seed=18)
    for i, mask in enumerate((-np.inf, torch.finfo(ref.TORCH[kind]).min, float("nan"))):
        l[i::4, 5] = mask
        l[i::8, 16:28] = mask  # a group of eight and half of the next
    l[47] = -np.inf
    b = randn(E, seed=19, std=0.1)
    b[[5, 22, 40]] = np.inf
    for groups in (1, 8):
        G, keep, gsum = GROUPS[groups]
        for renorm in (True, False):
            ids, w = run(l, kind, b, 10, score, n_group=G, top_group=keep, group_sum=gsum, renorm=renorm)
            assert np.isfinite(w).all()
    rising = torch.arange(32).float().repeat(3, 1) / 8
    rising[0, 5], rising[1, 5], rising[2, 5] = -np.inf, torch.finfo(ref.TORCH[kind]).min, float("nan")
    b = torch.zeros(32)
    b[5] = np.inf
    ids, _ = run(rising, kind, b, 3, score)
    assert (ids == [31, 30, 29]).all()


@pytest.mark.parametrize("score", [SOFT, SIG])
def test_groups_whose_sum_leaves_the_fp32_range(score):
    # three groups of four, the sums of the last two below fp32's lowest, and above its largest
    b = torch.zeros(12)
    b[4:8], b[8:] = -3e38, -2e38
    ids, _ = run(randn(8, 12, seed=20), qre.F32, b, 6, score, n_group=3, top_group=2, group_sum=2)
    assert (ids[:, :4] < 4).all() and (ids[:, 4:] >= 8).all()
    ids, _ = run(randn(8, 12, seed=20), qre.F32, -b, 6, score, n_group=3, top_group=2, group_sum=2)
    assert (ids[:, :4] // 4 == 1).all() and (ids[:, 4:] >= 8).all()
    # any finite biases, groups without a usable expert and with one
    l = randn(64, 64, seed=21)
    l[::3, 8:16] = -np.inf
    l[1::3, 17:24] = -np.inf
    low = -(torch.rand(64, generator=torch.Generator().manual_seed(22)) * 1.6 + 1.8) * 1e38
    for bias in (low, -low, torch.where(torch.arange(64) % 16 < 8, low, -low), torch.full((64,), torch.finfo(torch.float32).min)):
        for keep in (1, 3, 7, 8):
            run(l, qre.F32, bias, 8, score, n_group=8, top_group=keep, group_sum=2)


@pytest.mark.parametrize("ties", [2, 3, 5])
def test_ties_at_the_end_of_the_choice_hide_no_near_value(ties):
    """Equal experts on both sides of the end of the k, and another behind them whose value 32 bits cannot tell from theirs."""
    T, E = 400, 64
    g = np.random.default_rng(23)
    l = (np.full((T, E), -4.0) + g.uniform(-0.1, 0.1, (T, E))).astype(np.float32)
    b = g.uniform(-0.01, 0.01, E).astype(np.float32)
    b[:32] = b[0]
    for t in range(T):
        e = g.choice(32, ties, replace=False)
        l[t, e] = g.uniform(0.5, 2.0)
        other = g.integers(32, E)
        v = 1 / (1 + np.exp(-np.float64(l[t, e[0]]))) + np.float64(b[0]) - np.float64(b[other])
        l[t, other] = np.float32(np.log(v / (1 - v)))
        l[t, g.choice(np.setdiff1d(np.arange(E), [*e, other]), 2, replace=False)] = 6.0, 7.0
    lt, bt = torch.from_numpy(l), torch.from_numpy(b)
    for k in range(1, ties + 5):
        run(lt, qre.F32, bt, k, SIG)
    run(lt, qre.F32, bt, 3, SIG, n_group=8, top_group=8, group_sum=2)
    # under a softmax: equal largest experts without a bias, another's bias made to fit
    for t in range(60):
        row = g.uniform(-1, 1, E)
        e = np.sort(g.choice(E, ties + 1, replace=False))
        row[e[:ties]] = 1.5
        row = row.astype(np.float32)
        p = np.exp(row.astype(np.float64) - 1.5)
        p /= p.sum()
        bias = np.zeros(E, np.float32)
        bias[e[ties]] = np.float32(p[e[0]] - p[e[ties]])
        for k in range(1, ties + 1):
            run(torch.from_numpy(row[None]), qre.F32, torch.from_numpy(bias), k, SOFT)


def test_far_negative_sigmoids_keep_their_weights():
    """Scores down to the subnormal numbers, which the clamp of the sum raises by 2^14.  (Half a step of a subnormal, 2^-150, times that
    and the scale is inside run()'s 2^-126.)"""
    l = torch.linspace(-105, -60, 4 * 64).view(4, 64)
    for bias in (None, randn(64, seed=24, std=0.1)):
        for renorm in (True, False):
            for groups in (1, 8):
                G, keep, gsum = GROUPS[groups]
                run(l, qre.F32, bias, 10, SIG, n_group=G, top_group=keep, group_sum=gsum, renorm=renorm, scale=2.5)
    _, w = run(torch.full((2, 32), -87.5), qre.F32, None, 4, SIG)
    assert (w > 0).all()
