"""strata_moe_q4_experts against its formula in 64 bits: types, formats, lists with gaps, repeats and one expert for all, and the ids that
it refuses on the device."""
import itertools

import numpy as np
import pytest
import torch

import ops_reference as ref
import q4_reference as q4ref
import quantized_routed_expert_top10_gb300 as qre
from ops_reference import U

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
KINDS = (qre.F32, qre.BF16, qre.F16)


def rows(T, n, pad, kind, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(T, n + pad, generator=g).to(ref.TORCH[kind]).to(DEV)


class Layer:
    def __init__(self, E, d_model, d_ff, group=32, zeros=False, scale=qre.BF16, xk=qre.F32, ok=qre.F32, k=2, pad=0, apart=0, seed=1):
        self.E, self.k, self.xk, self.ok, self.pad = E, k, xk, ok, pad
        self.d_model, self.d_ff = d_model, d_ff
        self.gu = q4ref.Matrices(E, 2 * d_ff, d_model, group, zeros, scale, paired=True, seed=seed)
        self.dn = q4ref.Matrices(E, d_model, d_ff, group, zeros, scale, seed=seed + 1)
        self.pack(apart)

    def pack(self, apart=0):
        self.packed = []
        strides = []
        for m in (self.gu, self.dn):
            p = m.packed(DEV)
            wide = torch.full((self.E, p.shape[1] + apart), 0xFF, dtype=torch.uint8, device=DEV)
            wide[:, :p.shape[1]] = p
            self.packed.append(wide)
            strides.append(wide.shape[1])
        self.d = qre.q4_experts(self.gu.q, self.packed[0], self.dn.q, self.packed[1], self.E, self.k, self.xk, self.ok, strides[0],
                                strides[1], self.d_model + self.pad, self.d_model + 2 * self.pad)

    def workspace(self, T):
        ws = torch.full((qre.strata_moe_q4_experts_workspace_bytes(self.d, T),), 0xFF, dtype=torch.uint8, device=DEV)
        qre.strata_moe_workspace_init(ws)
        return ws

    def call(self, x, ids, weights, out, ws):
        qre.strata_moe_q4_experts(self.d, torch.as_tensor(ids, dtype=torch.int32, device=DEV),
                                  torch.as_tensor(weights, dtype=torch.float32, device=DEV), x, x.shape[0], out, ws)

    def check(self, ids, weights, seed=3, x=None):
        ids, weights = np.asarray(ids, np.int32), np.asarray(weights, np.float32)
        T = ids.shape[0]
        x = rows(T, self.d_model, self.pad, self.xk, seed) if x is None else x
        out = rows(T + 2, self.d_model, 2 * self.pad, self.ok, seed + 1)
        before, ws = out.clone(), self.workspace(T)
        self.call(x, ids, weights, out[1:], ws)
        assert qre.strata_poll_status(ws) == 0
        want, err = q4ref.experts(ref.to64(x[:, :self.d_model]), self.gu, self.dn, ids, weights.astype(np.float64), self.ok, self.xk)
        ref.check(out[1:T + 1, :self.d_model], want, err, self.ok, f"{T} tokens, {self.E} experts")
        out[1:T + 1, :self.d_model] = before[1:T + 1, :self.d_model]
        assert torch.equal(out.view(torch.uint8), before.view(torch.uint8))  # nothing beside the result


def lists(T, E, k, seed=1, distinct=True):
    host = np.random.RandomState(seed)
    ids = np.argsort(host.random_sample((T, E)), 1)[:, :k] if distinct else host.randint(0, E, (T, k))
    return ids.astype(np.int32), host.random_sample((T, k)).astype(np.float32) + 0.05


@pytest.mark.parametrize("xk,ok", list(itertools.product(KINDS, KINDS)))
@pytest.mark.parametrize("group,zeros", list(itertools.product((32, 64, 128), (False, True))))
def test_types(xk, ok, group, zeros):
    layer = Layer(6, 256, 128, group, zeros, qre.F16 if zeros else qre.BF16, xk, ok, k=3)
    layer.check(*lists(1, 6, 3))
    layer.check(*lists(5, 6, 3))


@pytest.mark.parametrize("T", [1, 2, 3, 4, 8, 9, 16, 17, 33, 64])
@pytest.mark.parametrize("xk,ok", [(qre.F32, qre.F32), (qre.BF16, qre.BF16)])
def test_tokens(T, xk, ok):
    layer = Layer(12, 128, 96, xk=xk, ok=ok, k=4)
    layer.check(*lists(T, 12, 4))


@pytest.mark.parametrize("d_model,d_ff,group", [(32, 32, 32), (32, 416, 32), (160, 32, 32), (1184, 416, 32), (2560, 640, 64), (192, 1088, 64),
                                                (128, 128, 128), (1408, 256, 128), (8192, 64, 32), (64, 8192, 64)])
def test_sizes(d_model, d_ff, group):
    for xk, ok, zeros in ((qre.F32, qre.F32, False), (qre.F16, qre.BF16, True)):
        layer = Layer(5, d_model, d_ff, group, zeros, xk=xk, ok=ok, k=2)
        layer.check(*lists(3, 5, 2))
        layer.check(*lists(1, 5, 2))


def test_one_expert_for_all():
    """All tokens at one expert: several blocks of columns over the same weights."""
    for xk, ok in ((qre.F32, qre.F32), (qre.BF16, qre.F16)):
        layer = Layer(3, 256, 128, xk=xk, ok=ok, k=1)
        layer.check(np.full((64, 1), 1), np.ones((64, 1)))
        Layer(1, 96, 64, xk=xk, ok=ok, k=1).check(np.zeros((7, 1)), np.full((7, 1), 0.5))


def test_many_experts():
    """More experts than pairs, the most experts and the longest lists."""
    Layer(1024, 64, 32, k=8).check(*lists(64, 1024, 8))
    Layer(40, 96, 32, k=32).check(*lists(64, 40, 32))
    Layer(512, 128, 64, k=10).check(*lists(1, 512, 10))


@pytest.mark.parametrize("group,zeros", list(itertools.product((32, 64), (False, True))))
def test_units_of_32_rows(group, zeros):
    """Enough experts and rows for units of two slabs."""
    scale = qre.F16 if zeros else qre.BF16
    Layer(128, 64, 512, group, zeros, scale, qre.BF16, qre.BF16, k=4).check(*lists(64, 128, 4))
    Layer(256, 192, 320, group, zeros, scale, qre.F32, qre.F32, k=4).check(*lists(60, 256, 4))
    Layer(200, 128, 512, group, zeros, scale, qre.F32, qre.F16, k=32).check(*lists(4, 200, 32))
    layer = Layer(256, 64, 448, group, zeros, scale, qre.F16, qre.BF16, k=4)
    ids, w = lists(64, 256, 4)
    ids[:40, 0] = 7  # one expert of many pairs among them: blocks over the same weights
    w[3] = 0.0
    layer.check(ids, w)


def test_the_same_expert_twice():
    Layer(4, 128, 64, k=5).check(*lists(9, 4, 5, distinct=False))
    Layer(4, 128, 64, k=3).check(np.full((4, 3), 2), np.full((4, 3), 0.3))


def test_slots_without_an_expert():
    layer = Layer(8, 128, 64, k=4)
    ids, w = lists(10, 8, 4)
    ids[0, :], w[1, :] = -1, 0.0
    ids[2, 1], w[3, 2], w[4, 0] = -1, 0.0, -0.0
    w[5, 3] = -0.7
    layer.check(ids, w)
    layer.check(np.full((3, 4), -1), np.ones((3, 4)))
    layer.check(np.zeros((3, 4)), np.zeros((3, 4)))


def test_nothing_of_an_expert_without_weight_is_read():
    """Experts that no token weighs hold scales of NaN."""
    layer = Layer(8, 128, 64, k=3)
    ids, w = lists(6, 4, 3)  # experts 0 .. 3
    w[:, 2] = 0.0
    ids[:, 2] = 5
    for m in (layer.gu, layer.dn):
        m.scales[4:] = float("nan")
    layer.pack()
    for m in (layer.gu, layer.dn):
        m.scales[4:] = 0.0  # for the formula
    layer.check(ids, w)


def test_strides():
    for ok in KINDS:
        Layer(5, 160, 96, xk=qre.BF16, ok=ok, pad=8, apart=48, k=3).check(*lists(7, 5, 3))


def test_single_products():
    """x with one column that is not 0, gate and up and down with one code a row that is not 8, so that no sum hides a term: gate and up
    are off by 10 u each (x has 22 bits: 4 u, and 6 roundings), the hidden value by 2 (the sigmoid's slope) * 10 + 10 + 8 = 38 u, the output by
    10 more and the weight's by 2."""
    E, d_model, d_ff = 2, 64, 32
    layer = Layer(E, d_model, d_ff, k=1)
    host = np.random.RandomState(3)
    q = np.full((E, d_model, d_ff), 8)
    for e in range(E):
        q[e, np.arange(d_model), host.randint(0, d_ff, d_model)] = host.choice([1, 3, 5, 11, 13, 15], d_model)
    layer.dn.set_codes(q)
    layer.pack()
    x = torch.diag(rows(1, d_model, 0, qre.F32, 4)[0])
    ids, w = host.randint(0, E, (d_model, 1)).astype(np.int32), np.ones((d_model, 1), np.float32)
    out, ws = torch.empty(d_model, d_model, device=DEV), layer.workspace(d_model)
    layer.call(x, ids, w, out, ws)
    want, _ = q4ref.experts(ref.to64(x), layer.gu, layer.dn, ids, w.astype(np.float64), qre.F32)
    got = ref.to64(out)
    assert (np.abs(got - want) <= 50 * U * np.abs(want)).all()


def test_rows_with_nan_and_infinities_stay_by_themselves():
    layer = Layer(4, 128, 64, k=2)
    ids, w = lists(30, 4, 2)
    x, ws = rows(30, 128, 0, qre.F32, 5), layer.workspace(30)
    clean, y = torch.empty(30, 128, device=DEV), torch.empty(30, 128, device=DEV)
    layer.call(x, ids, w, clean, ws)
    for r, v in ((3, float("nan")), (8, float("inf")), (29, 3.4e38)):
        x[r, 4 * r] = v
    layer.call(x, ids, w, y, ws)
    rest = [r for r in range(30) if r not in (3, 8, 29)]
    assert torch.equal(y[rest], clean[rest])
    assert not torch.isfinite(y[[3, 8]]).any()
    wn = w.copy()
    wn[5, 0] = np.nan
    x = torch.nan_to_num(x, posinf=0.0)
    layer.call(x, ids, wn, y, ws)
    assert torch.isnan(y[5]).all() and torch.isfinite(y[6]).all()


@pytest.mark.parametrize("bad", [-2, 4, 1 << 30, -(1 << 31)])
def test_bad_ids_compute_nothing(bad):
    layer = Layer(4, 128, 64, k=2)
    for T in (1, 30):
        ids, w = lists(T, 4, 2)
        x, ws = rows(T, 128, 0, qre.F32, 5), layer.workspace(T)
        out, again = rows(T, 128, 0, qre.F32, 6), torch.empty(T, 128, device=DEV)
        before, broken = out.clone(), ids.copy()
        broken[T - 1, 1] = bad
        layer.call(x, broken, w, out, ws)
        assert qre.strata_poll_status(ws) == -7
        assert torch.equal(out, before)
        qre.strata_clear_status(ws)
        layer.call(x, ids, w, out, ws)
        assert qre.strata_poll_status(ws) == 0
        layer.call(x, ids, w, again, layer.workspace(T))
        assert torch.equal(out, again)
        # also where the slot has no weight
        broken, w0 = ids.copy(), w.copy()
        broken[0, 0], w0[0, 0] = bad, 0.0
        out.copy_(before)
        layer.call(x, broken, w0, out, ws)
        assert qre.strata_poll_status(ws) == -7 and torch.equal(out, before)


def test_same_bits_again_in_graphs_and_on_streams():
    layer = Layer(16, 256, 128, k=4, xk=qre.BF16, ok=qre.F32)
    for T in (1, 40):
        ids, w = (torch.from_numpy(a).to(DEV) for a in lists(T, 16, 4))
        x, ws = rows(T, 256, 0, qre.BF16, 1), layer.workspace(T)
        y, z = torch.empty(T, 256, device=DEV), torch.empty(T, 256, device=DEV)
        layer.call(x, ids, w, y, ws)
        ws2 = layer.workspace(T)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(5):
                layer.call(x, ids, w, z, ws2)
        for _ in range(5):
            layer.call(x, ids, w, y, ws)  # at the same time
        torch.cuda.synchronize()
        assert torch.equal(y, z)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            qre.strata_moe_q4_experts(layer.d, ids, w, x, T, z, ws)
            qre.strata_moe_q4_experts(layer.d, ids, w, x, T, z, ws)
        new, wn = lists(T, 16, 4, seed=9)
        ids.copy_(torch.from_numpy(new))
        w.copy_(torch.from_numpy(wn))
        x.copy_(rows(T, 256, 0, qre.BF16, 2))
        g.replay()
        layer.call(x, ids, w, y, ws2)
        torch.cuda.synchronize()
        assert torch.equal(y, z)


def test_workspace_shared_with_a_decode_layer():
    """The scratch keeps clear of the words that other calls keep in a workspace."""
    from gpu_common import workspace
    layer = Layer(4, 128, 64, k=2)
    ids, w = lists(4, 4, 2)
    ws = workspace(64)
    assert ws.numel() >= qre.strata_moe_q4_experts_workspace_bytes(layer.d, 4)
    keep = ws[:1 << 20].clone()
    out = torch.empty(4, 128, device=DEV)
    layer.call(rows(4, 128, 0, qre.F32, 5), ids, w, out, ws)
    assert qre.strata_poll_status(ws) == 0
    assert torch.equal(ws[:1 << 20], keep)


def test_offsets_beyond_32_bits():
    """Experts and rows more than 2^32 bytes apart."""
    layer = Layer(3, 64, 32, k=2, xk=qre.BF16, ok=qre.BF16)
    ids, w = lists(5, 3, 2)
    x, want = rows(5, 64, 0, qre.BF16, 5), torch.empty(5, 64, dtype=torch.bfloat16, device=DEV)
    layer.call(x, ids, w, want, layer.workspace(5))
    step = (1 << 32) + 256
    big = torch.empty(4 * step + 65536, dtype=torch.uint8, device=DEV)
    for e in range(3):
        for i, p in enumerate(layer.packed):
            big[e * step + 8192 * i:e * step + 8192 * i + p.shape[1]] = p[e]
    assert max(p.shape[1] for p in layer.packed) <= 8192
    halves = big.view(torch.bfloat16)
    far_x, out = (torch.as_strided(halves, (5, 64), (step // 2, 1), at) for at in (10240, 12288))
    far_x.copy_(x)
    d = layer.d
    layer.d = qre.q4_experts(layer.gu.q, big.data_ptr(), layer.dn.q, big.data_ptr() + 8192, 3, 2, qre.BF16, qre.BF16, step, step,
                             step // 2, step // 2)
    ws = layer.workspace(5)
    qre.strata_moe_q4_experts(layer.d, torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV), far_x.data_ptr(), 5, out.data_ptr(), ws)
    assert qre.strata_poll_status(ws) == 0
    assert torch.equal(out, want)
    layer.d = d


def test_many_calls_in_a_row_on_one_workspace():
    """Token counts, shapes and lists change from call to call: the meetings' counters are 0 again after each."""
    layers = [Layer(6, 128, 64, k=2), Layer(9, 256, 96, k=3, xk=qre.BF16, ok=qre.BF16, zeros=True)]
    ws = torch.zeros(max(qre.strata_moe_q4_experts_workspace_bytes(x.d, 64) for x in layers), dtype=torch.uint8, device=DEV)
    for i in range(40):
        layer, T = layers[i % 2], (1, 5, 64, 2, 17)[i % 5]
        ids, w = lists(T, layer.E, layer.k, seed=i)
        x = rows(T, layer.d_model, 0, layer.xk, i)
        got, want = (torch.empty(T, layer.d_model, dtype=ref.TORCH[layer.ok], device=DEV) for _ in range(2))
        layer.call(x, ids, w, got, ws)
        layer.call(x, ids, w, want, layer.workspace(T))
        assert torch.equal(got, want), (i, T)
    assert qre.strata_poll_status(ws) == 0
    assert int(ws[8192:8192 + 12].sum()) == 0
