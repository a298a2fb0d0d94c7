"""strata_moe_linear against its formula in 64 bits: formats, types, sizes that end inside tiles, strides, and rows that must not touch
one another."""
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


def rows(T, n, pad, kind, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, n + pad, generator=g) * std).to(ref.TORCH[kind]).to(DEV)


class Bf16Rows:
    """bf16 weights with the interface of q4_reference.Matrices."""
    group = 128

    def __init__(self, n_out, d_in, pad=0, seed=1):
        self.n_out, self.d_in, self.pad = n_out, d_in, pad
        self.w = rows(n_out, d_in, pad, qre.BF16, seed, d_in ** -0.5)

    def weights(self, i):
        return ref.to64(self.w[:, :self.d_in])

    def descriptor(self, xk, yk, x_stride, y_stride):
        return qre.linear_bf16(self.w.data_ptr(), self.n_out, self.d_in, xk, yk, self.d_in + self.pad, x_stride, y_stride)


def check(m, T, xk=qre.F32, yk=qre.F32, bias=True, xpad=0, ypad=0, x=None, seed=3):
    x = rows(T, m.d_in, xpad, xk, seed) if x is None else x
    xpad = x.shape[1] - m.d_in
    y = rows(T + 2, m.n_out, ypad, yk, seed + 1)
    before = y.clone()
    b = rows(1, m.n_out, 0, qre.F32, seed + 2)[0] if bias else None
    if isinstance(m, Bf16Rows):
        keep, d = None, m.descriptor(xk, yk, m.d_in + xpad, m.n_out + ypad)
    else:
        keep = m.packed(DEV)
        d = qre.linear_q4(m.q, keep, xk, yk, m.d_in + xpad, m.n_out + ypad)
    qre.strata_moe_linear(d, x, T, b, y[1:])
    torch.cuda.synchronize()
    x64 = ref.to64(x[:, :m.d_in])
    x_err = np.zeros_like(x64) if isinstance(m, Bf16Rows) else q4ref.held(x64, 22 if xk == qre.F32 else 60)
    want, err = q4ref.product(x64, x_err, m.weights(0), q4ref.additions(m.d_in, m.group))
    if bias:
        want = want + ref.to64(b)
        err = err + U * np.abs(want)
    ref.check(y[1:T + 1, :m.n_out], want, err, yk, f"{T} x {m.d_in} -> {m.n_out}")
    y[1:T + 1, :m.n_out] = before[1:T + 1, :m.n_out]
    assert torch.equal(y.view(torch.uint8), before.view(torch.uint8))  # nothing beside the result
    del keep


@pytest.mark.parametrize("group,zeros", list(itertools.product((32, 64, 128), (False, True))))
@pytest.mark.parametrize("xk,yk", list(itertools.product(KINDS, KINDS)))
def test_types(group, zeros, xk, yk):
    scale = qre.F16 if zeros else qre.BF16
    check(q4ref.Matrices(1, 200, 640, group, zeros, scale), 1, xk, yk)
    check(q4ref.Matrices(1, 72, 2560, group, zeros, scale), 5, xk, yk, bias=False)


@pytest.mark.parametrize("xk,yk", list(itertools.product(KINDS, KINDS)))
def test_bf16_weights(xk, yk):
    check(Bf16Rows(512, 2560), 1, xk, yk)
    check(Bf16Rows(77, 328, pad=8), 9, xk, yk, xpad=8)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 7, 8, 9, 12, 13, 16, 17, 23, 24, 25, 33, 48, 64, 65, 200])
def test_tokens(T):
    for xk in KINDS:
        check(q4ref.Matrices(1, 100, 384, 64, True), T, xk, qre.F32)
        check(Bf16Rows(40, 200), T, xk, qre.F32)


@pytest.mark.parametrize("group,d_in", [(32, 32), (32, 64), (32, 96), (32, 160), (32, 1184), (64, 64), (64, 192), (64, 1088), (128, 128),
                                        (128, 2944)])
@pytest.mark.parametrize("n_out", [1, 15, 16, 17, 33])
def test_sizes(group, d_in, n_out):
    for zeros in (False, True):
        check(q4ref.Matrices(1, n_out, d_in, group, zeros), 3, qre.BF16, qre.F32)


@pytest.mark.parametrize("d_in", [8, 16, 24, 32, 40, 56, 64, 72, 136, 1000])
@pytest.mark.parametrize("n_out", [1, 15, 16, 17, 33])
def test_bf16_sizes(d_in, n_out):
    check(Bf16Rows(n_out, d_in), 2, qre.F32, qre.F32)


@pytest.mark.parametrize("n_out,d_in,T", [(2432, 256, 1), (2433, 256, 2), (4864, 1280, 1), (9728, 128, 3), (19457, 128, 1), (40000, 64, 2)])
def test_many_rows(n_out, d_in, T):
    """From one unit of 16 rows a CTA to several for each of its warps."""
    check(q4ref.Matrices(1, n_out, d_in, 64), T, qre.BF16, qre.BF16)
    check(Bf16Rows(n_out, d_in), T, qre.BF16, qre.F32)


@pytest.mark.parametrize("n_out", [77823, 77825, 77840, 77856, 100001])
def test_units_of_32_rows(n_out):
    """Enough rows for units of two slabs, an odd number of slabs, and one slab less."""
    for group, d_in, T, xk, zeros in ((32, 96, 1, qre.F32, True), (64, 320, 3, qre.BF16, False), (128, 256, 4, qre.F32, True), (32, 32, 8, qre.F16, False)):
        check(q4ref.Matrices(1, n_out, d_in, group, zeros, qre.F16 if zeros else qre.BF16), T, xk, qre.F32)


@pytest.mark.parametrize("T,xk,d_in", [(64, qre.F32, 2560), (24, qre.BF16, 8192), (8, qre.F32, 16384), (1, qre.F32, 32768), (3, qre.F32, 28672),
                                       (30, qre.F16, 4096)])
def test_activations_in_panels(T, xk, d_in):
    """Columns that do not all lie in shared memory at once."""
    check(q4ref.Matrices(1, 40, d_in, 128, True), T, xk, qre.F32)
    check(q4ref.Matrices(1, 2500, d_in, 32), T, xk, qre.F32)
    check(Bf16Rows(40, d_in), T, xk, qre.F32)


@pytest.mark.parametrize("T,xk,d_in,n_out", [(24, qre.BF16, 1408, 32), (24, qre.F16, 1440, 33), (25, qre.BF16, 2560, 2432), (33, qre.F16, 1376, 2416),
                                             (64, qre.BF16, 2560, 10240), (65, qre.BF16, 2592, 10241), (12, qre.F32, 1440, 512), (13, qre.F32, 1408, 496),
                                             (200, qre.F32, 1472, 48), (64, qre.F32, 1440, 4880), (4000, qre.BF16, 1408, 40)])
def test_activations_laid_out_by_two(T, xk, d_in, n_out):
    """Enough of x for neighbouring CTAs to share its layout, with last blocks of one token, even and odd numbers of units."""
    check(q4ref.Matrices(1, n_out, d_in, 32, True, qre.BF16), T, xk, qre.F32)


@pytest.mark.parametrize("T,xk", [(24, qre.BF16), (25, qre.BF16), (12, qre.F16), (49, qre.F16), (8, qre.F32), (17, qre.F32)])
@pytest.mark.parametrize("n_out", [32, 497])
def test_activations_of_bf16_rows_laid_out_by_two(T, xk, n_out):
    check(Bf16Rows(n_out, 1416), T, xk, qre.F32)


def test_layout_by_two_again_in_graphs_and_beside_others():
    m = q4ref.Matrices(1, 2560, 2560, 64, False, qre.BF16)
    keep = m.packed(DEV)
    d = qre.linear_q4(m.q, keep, qre.BF16, qre.BF16)
    streams = [torch.cuda.Stream() for _ in range(3)]
    x = [rows(64, 2560, 0, qre.BF16, 11 + i) for i in range(3)]
    y = [rows(64, 2560, 0, qre.BF16, 21 + i) for i in range(3)]
    for i in range(3):
        qre.strata_moe_linear(d, x[i], 64, None, y[i])
    torch.cuda.synchronize()
    want = [v.clone() for v in y]
    for v in y:
        v.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                qre.strata_moe_linear(d, x[i], 64, None, y[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(y, want))
    for v in y:
        v.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for i in range(3):
            qre.strata_moe_linear(d, x[i], 64, None, y[i])
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(y, want))


@pytest.mark.parametrize("yk", KINDS)
def test_strides(yk):
    check(q4ref.Matrices(1, 51, 320, 64), 6, qre.F16, yk, xpad=24, ypad=3)
    check(Bf16Rows(51, 320, pad=16), 6, qre.BF16, yk, xpad=24, ypad=3)


@pytest.mark.parametrize("bf16", [False, True])
def test_single_products_are_exact_to_their_rounding(bf16):
    """One column of x holds a number of 24 bits and the others 0: every weight by itself, in its place.  Products of terms are
    exact, each is scaled and added: 6 roundings (the scale's product, two additions of terms, the sums of zeros none); beside 4-bit
    weights x itself is off by 2^-22 = 4 u."""
    d_in, n_out = 320, 48
    m = Bf16Rows(n_out, d_in) if bf16 else q4ref.Matrices(1, n_out, d_in, 32, True)
    keep = None if bf16 else m.packed(DEV)
    d = m.descriptor(qre.F32, qre.F32, d_in, n_out) if bf16 else qre.linear_q4(m.q, keep)
    value = rows(1, d_in, 0, qre.F32, 9)[0]
    x, y = torch.diag(value), torch.empty(d_in, n_out, device=DEV)
    qre.strata_moe_linear(d, x, d_in, None, y)
    want = ref.to64(value)[:, None] * m.weights(0).T
    got = ref.to64(y)
    assert (np.abs(got - want) <= (6 if bf16 else 10) * U * np.abs(want)).all()


def test_rows_with_nan_and_infinities_stay_by_themselves():
    m = q4ref.Matrices(1, 64, 256, 64)
    packed, bf = m.packed(DEV), Bf16Rows(64, 256)
    for d, w in ((qre.linear_q4(m.q, packed), m.weights(0)), (bf.descriptor(qre.F32, qre.F32, 256, 64), None)):
        x = rows(20, 256, 0, qre.F32, 5)
        clean, y = torch.empty(20, 64, device=DEV), torch.empty(20, 64, device=DEV)
        qre.strata_moe_linear(d, x, 20, None, clean)
        for r, v in ((3, float("nan")), (8, float("inf")), (19, 3.4e38)):
            x[r, 7 * r] = v
        qre.strata_moe_linear(d, x, 20, None, y)
        rest = [r for r in range(20) if r not in (3, 8, 19)]
        assert torch.equal(y[rest], clean[rest])
        assert not torch.isfinite(y[[3, 8]]).any()
        if w is None:  # 3.4e38 rounds to bf16's infinity
            assert not torch.isfinite(y[19]).any()
        else:          # beside 4-bit weights it is a number like any other
            x64 = ref.to64(x[19:])
            want, err = q4ref.product(x64, q4ref.held(x64, 22), w, q4ref.additions(256, 64))
            ref.check(y[19:], want, err, qre.F32, "the largest numbers")


def test_same_bits_again_in_graphs_and_on_streams():
    m = q4ref.Matrices(1, 2600, 1280, 32, True)
    packed = m.packed(DEV)
    for T in (1, 20):
        d = qre.linear_q4(m.q, packed, qre.F32, qre.F32)
        x, y, z = rows(T, 1280, 0, qre.F32, 1), torch.empty(T, 2600, device=DEV), torch.empty(T, 2600, device=DEV)
        qre.strata_moe_linear(d, x, T, None, y)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(3):
                qre.strata_moe_linear(d, x, T, None, z)
        s.synchronize()
        assert torch.equal(y, z)
        g = torch.cuda.CUDAGraph()
        z.zero_()
        with torch.cuda.graph(g):
            qre.strata_moe_linear(d, x, T, None, z)
        x.copy_(rows(T, 1280, 0, qre.F32, 2))
        g.replay()
        qre.strata_moe_linear(d, x, T, None, y)
        torch.cuda.synchronize()
        assert torch.equal(y, z)


def test_weights_packed_on_the_host_and_on_the_device_agree():
    for group, zeros, paired in itertools.product((32, 64, 128), (False, True), (False, True)):
        m = q4ref.Matrices(3, 112, 640 if group == 128 else 320, group, zeros, paired=paired)
        assert torch.equal(m.packed(DEV).cpu(), m.packed_host())
        # codes on any byte
        odd = torch.empty(m.codes.numel() + 1, dtype=torch.uint8, device=DEV)
        odd[1:] = m.codes.flatten().to(DEV)
        to = torch.empty(3, qre.strata_q4_bytes(m.q), dtype=torch.uint8, device=DEV)
        qre.strata_pack_q4_device(m.q, odd[1:], m.scales.to(DEV), None if m.zeros is None else m.zeros.to(DEV), to, 3)
        assert torch.equal(to.cpu(), m.packed_host())


def test_packing_then_using_the_weights_at_once():
    """The call after the packing on the same stream sees the packed weights."""
    m = q4ref.Matrices(1, 4096, 2048, 64)
    codes, scales = m.codes.to(DEV), m.scales.to(DEV)
    x = rows(1, 2048, 0, qre.F32, 1)
    want = torch.empty(1, 4096, device=DEV)
    packed = m.packed(DEV)
    qre.strata_moe_linear(qre.linear_q4(m.q, packed), x, 1, None, want)
    torch.cuda.synchronize()
    for _ in range(5):
        y, packed = torch.empty(1, 4096, device=DEV), torch.zeros_like(packed)
        torch.cuda.synchronize()
        qre.strata_pack_q4_device(m.q, codes, scales, None, packed)
        qre.strata_moe_linear(qre.linear_q4(m.q, packed), x, 1, None, y)
        assert torch.equal(y, want)


def test_offsets_beyond_32_bits():
    """Rows of x, y and bf16 weights more than 2^32 bytes apart."""
    step = (1 << 30) + 8
    big = torch.empty(4 * step + 4096, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(DEV).manual_seed(3)
    x = torch.as_strided(big, (5, 64), (step, 1))
    x.copy_(torch.randn(5, 64, generator=g, device=DEV))
    want_x = x.clone()
    for n_out, w in ((40, None), (5, torch.as_strided(big, (5, 64), (step, 1), 256))):
        y = torch.as_strided(big, (5, n_out), (step, 1), 1024)
        if w is None:
            m = q4ref.Matrices(1, n_out, 64, 32)
            packed = m.packed(DEV)
            d = qre.linear_q4(m.q, packed, qre.BF16, qre.BF16, step, step)
            dense = qre.linear_q4(m.q, packed, qre.BF16, qre.BF16)
        else:
            w.copy_(torch.randn(5, 64, generator=g, device=DEV))
            rows_w = w.contiguous()
            d = qre.linear_bf16(w.data_ptr(), n_out, 64, qre.BF16, qre.BF16, step, step, step)
            dense = qre.linear_bf16(rows_w, n_out, 64, qre.BF16, qre.BF16)
        want = torch.empty(5, n_out, dtype=torch.bfloat16, device=DEV)
        qre.strata_moe_linear(d, x.data_ptr(), 5, None, y.data_ptr())
        qre.strata_moe_linear(dense, want_x, 5, None, want)
        assert torch.equal(y, want)


def test_on_a_stream_beside_others():
    """Calls of two streams at once, each with its own rows."""
    m = q4ref.Matrices(1, 3000, 1024, 128)
    packed = m.packed(DEV)
    d = qre.linear_q4(m.q, packed)
    xs = [rows(T, 1024, 0, qre.F32, T) for T in (1, 7, 30)]
    want = [torch.empty(x.shape[0], 3000, device=DEV) for x in xs]
    got = [torch.empty_like(w) for w in want]
    for x, w in zip(xs, want):
        qre.strata_moe_linear(d, x, x.shape[0], None, w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(10):
        for s, x, y in zip(streams, xs, got):
            qre.strata_moe_linear(d, x, x.shape[0], None, y, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
