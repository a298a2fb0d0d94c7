"""strata_moe_norm and strata_moe_combine_norm against their formulas in 64 bits."""
import itertools

import numpy as np
import pytest
import torch

import ops_reference as ref
import quantized_routed_expert_top10_gb300 as qre

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
KINDS = (qre.F32, qre.BF16, qre.F16)


def rnd(*shape, seed=0, std=1.0, mean=0.0, kind=qre.F32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std + mean).to(ref.TORCH[kind]).to(DEV)


def padded(T, n, stride, kind, seed=0, offset=0, std=1.0):
    """A [T][n] view of rows `stride` elements apart that starts `offset` elements into its buffer, and the buffer."""
    buf = rnd(T * stride + offset, seed=seed, kind=kind, std=std)
    return buf[offset:offset + T * stride].view(T, stride)[:, :n], buf


def run_norm(T, n, xk, ok, gain=True, pad=0, offset=0, eps=1e-6, inplace=False, x=None):
    stride = n + pad
    xv, _ = padded(T, n, stride, xk, seed=n, offset=offset)
    if x is not None:
        xv.copy_(x)
    before = ref.to64(xv)
    ov, obuf = (xv, None) if inplace else padded(T, n, stride, ok, seed=99, offset=offset)
    keep = None if obuf is None else obuf.clone()
    gv = rnd(n, seed=3, std=0.2, mean=1.0) if gain else None
    d = qre.norm(n, eps, xk, ok, stride, stride)
    qre.strata_moe_norm(d, xv.data_ptr(), T, gv, ov.data_ptr())
    torch.cuda.synchronize()
    want, err = ref.rms_norm(before, np.zeros_like(before), eps, None if gv is None else ref.to64(gv))
    ref.check(ov, want, err, ok, "norm")
    if obuf is not None and obuf.numel() > T * n:  # nothing beside the rows was written
        inside = torch.zeros_like(obuf, dtype=torch.bool)
        inside[offset:offset + T * stride].view(T, stride)[:, :n] = True
        assert torch.equal(obuf[~inside], keep[~inside])


@pytest.mark.parametrize("xk,ok", list(itertools.product(KINDS, KINDS)))
def test_norm_types(xk, ok):
    run_norm(5, 2560, xk, ok)


@pytest.mark.parametrize("n", [1, 2, 7, 8, 31, 64, 256, 264, 1000, 1001, 2560, 4096, 4104, 5120, 8192, 8200, 16376, 16383, 16384])
def test_norm_widths(n):
    for T in (1, 9):
        run_norm(T, n, qre.F32, qre.F32)
    run_norm(3, n, qre.BF16, qre.BF16, gain=False)


@pytest.mark.parametrize("T", [1, 4, 151, 304, 1000, 8192])
def test_norm_lengths(T):
    run_norm(T, 2560, qre.F32, qre.BF16)
    run_norm(T, 96, qre.F16, qre.F32)


def test_norm_strides_alignment_and_in_place():
    for n, pad, off in ((2560, 8, 0), (2560, 5, 0), (2560, 0, 1), (2560, 8, 3), (777, 0, 0), (64, 3, 5), (200, 8, 8)):
        for kind in KINDS:
            run_norm(7, n, kind, kind, pad=pad, offset=off)
            run_norm(7, n, kind, kind, pad=pad, offset=off, inplace=True)


def test_norm_rows_of_zeros_and_large_values():
    x = torch.zeros(4, 2560)
    x[1] = 1e-12
    x[2] = 1e15
    x[3, 7] = -3.0
    run_norm(4, 2560, qre.F32, qre.F32, x=x.to(DEV))
    run_norm(4, 2560, qre.F32, qre.F32, x=x.to(DEV), eps=1e-2)


def run_edge(T, n, P, pk=qre.F32, xk=qre.F32, nk=qre.F32, post=True, gain=True, channel=True, token="sigmoid", weights=True,
             x=True, out=True, nxt=True, pre=True, residual=0.9, block=0.5, pad=0, offset=0, inplace=None, zero_weight=False,
             eps=1e-6):
    ps = n + pad
    ts = P * ps + pad
    pbuf = rnd(T * ts + offset, seed=P + n, kind=pk)
    parts = torch.as_strided(pbuf, (T, P, n), (ts, ps, 1), offset)
    pw = torch.softmax(rnd(T, P, seed=2), 1) if weights else None
    if zero_weight:  # what a part of weight 0 holds does not matter
        pw[:, 0] = 0.0
        parts[:, 0] = float("nan")
        pw[0] = 0.0
        parts[0] = float("inf")
    xs = n + pad
    xv = padded(T, n, xs, xk, seed=4, offset=offset)[0] if x else None
    x64 = ref.to64(xv) if x else None
    ov = None if not out else xv if inplace == "out" else padded(T, n, xs, xk, seed=5, offset=offset)[0]
    nv = None if not nxt else xv if inplace == "next" else padded(T, n, xs, nk, seed=6, offset=offset)[0]
    post_gain = rnd(n, seed=7, std=0.1, mean=1.0) if post and gain else None
    ch = rnd(n, seed=8, std=0.3, mean=0.7) if channel else None
    tk = rnd(T, seed=9, std=2.0) if token else None
    pre_gain = rnd(n, seed=10, std=0.1, mean=1.0) if pre and nxt else None
    d = qre.combine_norm(n, P, post, token == "sigmoid", eps, residual, block, pk, xk, nk, ps, ts, xs, xs, xs)
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    qre.strata_moe_combine_norm(d, parts.data_ptr(), pw, ptr(xv), T, post_gain, ch, tk, pre_gain, ptr(ov), ptr(nv))
    torch.cuda.synchronize()
    h = lambda t: None if t is None else ref.to64(t)  # noqa: E731
    r, r_err, nx, nx_err = ref.edge(h(parts), h(pw), x64, post, h(post_gain), h(ch), h(tk), token == "sigmoid", h(pre_gain),
                                    eps, residual, block)
    if out:
        ref.check(ov, r, r_err, xk, "out")
    if nxt:
        ref.check(nv, nx, nx_err, nk, "next")


@pytest.mark.parametrize("pk,xk,nk", list(itertools.product(KINDS, KINDS, KINDS)))
def test_edge_types(pk, xk, nk):
    run_edge(3, 2560, 10, pk, xk, nk)


@pytest.mark.parametrize("n", [1, 7, 8, 64, 256, 264, 1000, 1001, 2560, 4104, 8200, 16383, 16384])
@pytest.mark.parametrize("P", [1, 3, 10])
def test_edge_widths(n, P):
    run_edge(2, n, P)
    run_edge(9, n, P, xk=qre.BF16, nk=qre.BF16)


@pytest.mark.parametrize("P", [1, 2, 4, 5, 9, 11, 16, 31, 32])
def test_edge_part_counts(P):
    run_edge(3, 2560, P, zero_weight=True)
    run_edge(3, 640, P, weights=False)


@pytest.mark.parametrize("T", [1, 2, 16, 151, 305, 2048])
def test_edge_lengths(T):
    run_edge(T, 2560, 10)


@pytest.mark.parametrize("n", [1, 3, 97, 255, 2559, 4097, 8193])
@pytest.mark.parametrize("T", [1, 152, 700, 2000])
def test_odd_rows_of_long_calls(n, T):
    """Rows off every boundary, more of them than are in flight at once."""
    T = min(T, 2000 * 2560 // n)
    run_norm(T, n, qre.F32, qre.BF16)
    run_norm(T, n, qre.BF16, qre.F16, pad=2, offset=1)
    run_edge(T, n, 3, qre.BF16, qre.F32, qre.F16, zero_weight=T > 1)
    run_edge(T, n, 1, qre.F32, qre.BF16, qre.BF16, offset=1, x=n % 2 == 0)
    run_edge(T, n, 2, qre.F16, qre.F16, qre.F32, pad=1, inplace="out", weights=False)


@pytest.mark.parametrize("n,T", [(64, 4000), (640, 1500), (4096, 400), (4100, 400), (8192, 300), (16384, 160)])
def test_aligned_rows_of_long_calls(n, T):
    run_norm(T, n, qre.F32, qre.F32, inplace=True)
    run_norm(T, n, qre.F16, qre.F32)
    run_edge(T, n, 3, qre.BF16, qre.F32, qre.F16, zero_weight=True)
    run_edge(T, n, 1, qre.F16, qre.BF16, qre.F32, inplace="out")
    run_edge(T, n, 2, qre.F32, qre.F16, qre.BF16, x=False)


def test_edge_largest_call():
    run_edge(8192, 2560, 1, xk=qre.BF16, nk=qre.BF16)


def test_edge_options():
    for post, gain, channel, token, weights, x in itertools.product((0, 1), (0, 1), (0, 1), (None, "raw", "sigmoid"), (0, 1), (0, 1)):
        run_edge(2, 320, 3, post=bool(post), gain=bool(gain), channel=bool(channel), token=token, weights=bool(weights), x=bool(x))
    run_edge(4, 2560, 10, out=False)
    run_edge(4, 2560, 10, nxt=False)
    run_edge(4, 2560, 10, pre=False)
    run_edge(4, 2560, 10, residual=0.0, block=-2.0, eps=0.0)


def test_edge_strides_alignment_and_in_place():
    for n, pad, off in ((2560, 8, 0), (2560, 5, 0), (2560, 0, 1), (777, 0, 0), (64, 3, 5), (200, 8, 8)):
        for kind in KINDS:
            run_edge(5, n, 4, kind, kind, kind, pad=pad, offset=off)
            run_edge(5, n, 4, kind, kind, kind, pad=pad, offset=off, inplace="out")
            run_edge(5, n, 4, kind, kind, kind, pad=pad, offset=off, inplace="next")


def test_edge_all_parts_masked_gives_the_residual():
    n = 2560
    x = rnd(2, n, seed=1)
    out = torch.empty_like(x)
    parts = torch.full((2, 10, n), float("nan"), device=DEV)
    qre.strata_moe_combine_norm(qre.combine_norm(n, 10), parts, torch.zeros(2, 10, device=DEV), x, 2, None, None, None, None,
                                out, None)
    torch.cuda.synchronize()
    assert torch.equal(out, x)


def test_repeats_streams_and_graphs():
    T, n = 37, 2560
    parts, pw, x = rnd(T, 10, n, seed=1), torch.softmax(rnd(T, 10, seed=2), 1), rnd(T, n, seed=3)
    out, nxt = torch.empty_like(x), torch.empty_like(x)
    d = qre.combine_norm(n, 10)

    def call():
        qre.strata_moe_combine_norm(d, parts, pw, x, T, None, None, None, None, out, nxt)

    call()
    torch.cuda.synchronize()
    first = out.clone(), nxt.clone()
    out.zero_(), nxt.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    assert torch.equal(out, first[0]) and torch.equal(nxt, first[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        qre.strata_moe_norm(qre.norm(n), out, T, None, nxt)  # in the graph, the norm reads what the call before it wrote
    x.copy_(rnd(T, n, seed=11))
    graph.replay()
    torch.cuda.synchronize()
    call()
    torch.cuda.synchronize()
    want, err = ref.rms_norm(ref.to64(out), np.zeros((T, n)), 1e-6, None)
    ref.check(nxt, want, err, qre.F32, "next")


def test_column_ranges_of_one_buffer():
    """Rows of one operand between the rows of another, as column ranges of one buffer: no element is shared."""
    for n, T in ((64, 5), (2560, 300), (100, 700), (77, 9)):
        def halves(seed, kind=qre.F32, count=2):
            buf = rnd(T, count * n, seed=seed, kind=kind)
            return buf, [buf[:, i * n:(i + 1) * n] for i in range(count)]

        for kind in KINDS:
            buf, (x, out) = halves(13, kind)
            want = torch.empty(T, n, dtype=x.dtype, device=DEV)
            before = x.clone()
            qre.strata_moe_norm(qre.norm(n, x_type=kind, out_type=kind), before, T, None, want)
            qre.strata_moe_norm(qre.norm(n, x_type=kind, out_type=kind, x_stride=2 * n, out_stride=2 * n), x.data_ptr(), T, None,
                                out.data_ptr())
            assert torch.equal(out, want) and torch.equal(x, before)
        # a combine's two parts, its x and both results
        buf, cols = halves(14, count=5)
        parts, x = buf[:, :2 * n].contiguous(), cols[2].contiguous()
        want = [torch.empty(T, n, device=DEV) for _ in range(2)]
        qre.strata_moe_combine_norm(qre.combine_norm(n, 2), parts, None, x, T, None, None, None, None, *want)
        qre.strata_moe_combine_norm(qre.combine_norm(n, 2, part_stride=n, token_stride=5 * n, x_stride=5 * n, out_stride=5 * n,
                                                     next_stride=5 * n), buf, None, cols[2].data_ptr(), T, None, None, None, None,
                                    cols[3].data_ptr(), cols[4].data_ptr())
        assert torch.equal(cols[3], want[0]) and torch.equal(cols[4], want[1])
        assert torch.equal(buf[:, :2 * n], parts) and torch.equal(cols[2], x)
        # a result in the gap between a token's two parts
        buf, (p0, gap, p1) = halves(15, count=3)
        parts = torch.cat([p0, p1], 1)
        qre.strata_moe_combine_norm(qre.combine_norm(n, 2), parts, None, None, T, None, None, None, None, want[0], None)
        qre.strata_moe_combine_norm(qre.combine_norm(n, 2, part_stride=2 * n, token_stride=3 * n, out_stride=3 * n), buf, None,
                                    None, T, None, None, None, None, gap.data_ptr(), None)
        assert torch.equal(gap, want[0]) and torch.equal(torch.cat([p0, p1], 1), parts)


def test_rows_without_a_mean_square_at_eps_0():
    """eps 0: a row of zeros, or whose squares vanish in fp32, is divided by 0; the rows beside it are not touched by that."""
    for n in (2560, 2559, 64):
        x = torch.randn(6, n, generator=torch.Generator().manual_seed(12))
        x[1] = 0.0
        x[3] = 1e-30 * torch.sign(x[3])
        x[3, ::2] = 0.0
        x[5] = 1e-12 * x[5]
        x = x.to(DEV)
        out, nxt = torch.empty_like(x), torch.empty_like(x)
        qre.strata_moe_norm(qre.norm(n, 0.0), x, 6, None, out)
        for P in (1, 2):  # the norm of the block's output is the same one; a token whose parts are all masked is a row of zeros
            parts = torch.zeros(6, P, n, device=DEV)
            parts[:, 0] = x
            pw = torch.zeros(6, P, device=DEV)
            pw[[0, 3, 5], 0] = 1.0
            qre.strata_moe_combine_norm(qre.combine_norm(n, P, eps=0.0), parts, pw, None, 6, None, None, None, None, nxt, None)
            torch.cuda.synchronize()
            assert nxt[[1, 2, 4]].isnan().all()
            for v in ((out, nxt) if P == 1 else (nxt,)):
                assert v[1].isnan().all() and v[3, ::2].isnan().all()
                assert torch.equal(v[3, 1::2], torch.sign(x[3, 1::2]) * np.inf)
                want, err = ref.rms_norm(ref.to64(x[[0, 5]]), np.zeros((2, n)), 0.0, None)
                ref.check(v[[0, 5]], want, err, qre.F32, "norm")
