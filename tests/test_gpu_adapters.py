"""strata_moe_adapters against its formula in 64 bits: ragged segments, every type, ranks and widths, in place, and the
segments that it refuses on the device."""
import itertools

import numpy as np
import pytest
import torch

import ops_reference as ref
import quantized_routed_expert_top10_gb300 as qre
from gpu_common import workspace

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
KINDS = (qre.F32, qre.BF16, qre.F16)


def rnd(*shape, seed=0, std=1.0, kind=qre.F32):
    g = torch.Generator(DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(ref.TORCH[kind])


def rows(T, n, stride, kind, seed):
    return torch.as_strided(rnd(T * stride, seed=seed, kind=kind), (T, n), (stride, 1))


class Case:
    def __init__(self, lens, of, rank, d_in, d_out, xk=qre.F32, yk=qre.F32, n=5, pad=0, before=0, after=0, base=True,
                 inplace=False, scale=True, seed=1, wpad=0):
        self.off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32) + before
        self.of = np.asarray(of, np.int32)
        self.T = int(self.off[-1]) + after
        self.rank, self.xk, self.yk = rank, xk, yk
        self.x = rows(self.T, d_in, d_in + pad, xk, seed)
        self.y = rows(self.T, d_out, d_out + pad, yk, seed + 1)
        self.base = self.y if inplace else rows(self.T, d_out, d_out + 2 * pad, yk, seed + 2) if base else None
        ast, bst = rank * d_in + wpad, rank * d_out + wpad
        self.a = torch.as_strided(rnd(n * ast, seed=seed + 3, std=d_in ** -0.5, kind=qre.BF16), (n, rank, d_in), (ast, d_in, 1))
        self.b = torch.as_strided(rnd(n * bst, seed=seed + 4, std=rank ** -0.5, kind=qre.BF16), (n, d_out, rank), (bst, rank, 1))
        self.scale = rnd(n, seed=seed + 5) if scale else None
        self.d = qre.adapters(self.a.data_ptr(), self.b.data_ptr(), n, rank, d_in, d_out, self.scale, xk, yk, ast, bst,
                              d_in + pad, d_out + (pad if inplace else 2 * pad), d_out + pad)
        self.d_in = d_in
        self.dev_off, self.dev_of = torch.from_numpy(self.off).to(DEV), torch.from_numpy(self.of).to(DEV)
        self.ws = workspace(self.T)

    def call(self):
        qre.strata_moe_adapters(self.d, self.dev_off, self.dev_of, len(self.of), self.x.data_ptr(), self.T,
                                None if self.base is None else self.base.data_ptr(), self.y.data_ptr(), self.ws)

    def check(self):
        y0 = ref.to64(self.y)
        base = None if self.base is None else ref.to64(self.base)
        before = self.y.clone()
        self.call()
        assert qre.strata_poll_status(self.ws) == 0
        want, delta = ref.adapters(ref.to64(self.x), ref.to64(self.a), ref.to64(self.b),
                                   None if self.scale is None else ref.to64(self.scale), self.off, self.of, base, y0)
        got = ref.to64(self.y)
        assert np.isfinite(got).all()
        lo, hi = self.off[0], self.off[-1]
        assert torch.equal(self.y[:lo], before[:lo]) and torch.equal(self.y[hi:], before[hi:])
        # the product's error by rows as 2-norms, the sum's and the result's rounding value by value
        err = np.maximum(np.abs(got - want) - (ref.half_step(self.yk) + ref.U) * np.abs(want), 0.0)
        row = np.sqrt(np.square(err).sum(1))
        room = ref.adapters_rtol(self.d_in, self.rank, self.yk) * np.sqrt(np.square(delta).sum(1)) * 2 + 1e-30
        if self.yk == qre.F16:
            room = room + 2.0 ** -24 * np.sqrt(got.shape[1])
        assert (row <= room).all(), (np.max(row / room), int(np.argmax(row / room)))
        none = [i for i, ad in enumerate(self.of) if ad < 0]
        for i in none:  # no adapter: the base itself
            s = slice(self.off[i], self.off[i + 1])
            if self.base is not None:
                assert torch.equal(self.y[s], before[s] if self.base is self.y else self.base[s])
            else:
                assert (self.y[s] == 0).all()


RAGGED = ([0, 1, 16, 17, 33, 0, 5, 64, 2, 0], [3, 0, 1, -1, 2, -1, 4, 2, 0, 0])


@pytest.mark.parametrize("xk,yk", list(itertools.product(KINDS, KINDS)))
def test_types(xk, yk):
    Case(*RAGGED, 16, 2560, 512, xk, yk).check()
    Case([1], [2], 16, 2560, 2560, xk, yk).check()


@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 56, 64, 72, 96, 120, 128])
def test_ranks(rank):
    Case(*RAGGED, rank, 320, 264).check()
    Case(*RAGGED, rank, 1000, 96, qre.BF16, qre.BF16).check()
    Case([300], [1], rank, 640, 640, qre.BF16, qre.F32).check()


LONG = ([200, 0, 130, 128, 1, 127, 70, 300], [3, 0, 1, -1, 2, 4, 2, 0])


@pytest.mark.parametrize("xk,yk", list(itertools.product(KINDS, KINDS)))
@pytest.mark.parametrize("rank", [8, 16, 40, 64, 72, 128])
def test_long_segments(xk, yk, rank):
    Case(*LONG, rank, 520, 392, xk, yk, before=1, after=3).check()
    Case([129, 300], [1, 1], rank, 2560, 1096, xk, yk, base=False).check()
    Case(*LONG, rank, 64, 2560, xk, yk, inplace=True, pad=8).check()


MANY = ([700, 0, 300, 128, 1, 127, 900, 250], [3, 0, 1, -1, 2, 4, 2, 0])  # 2,406 tokens


@pytest.mark.parametrize("xk,yk", list(itertools.product(KINDS, KINDS)))
@pytest.mark.parametrize("rank", [88, 96, 120, 128])
def test_many_tokens_and_ranks(xk, yk, rank):
    Case(*MANY, rank, 264, 392, xk, yk, before=1, after=3).check()
    Case(*MANY, rank, 64, 264, xk, yk, inplace=True, pad=8).check()


@pytest.mark.parametrize("xk,yk", [(qre.BF16, qre.BF16), (qre.F16, qre.F32), (qre.BF16, qre.F32), (qre.F16, qre.F16)])
@pytest.mark.parametrize("rank", [40, 56, 64, 72])
def test_many_tokens(xk, yk, rank):
    Case([2000, 127, 0, 2049, 1, 900], [0, 4, 1, 2, -1, 0], rank, 264, 136, xk, yk, after=2).check()


@pytest.mark.parametrize("xk,yk", list(itertools.product(KINDS, KINDS)))
@pytest.mark.parametrize("rank", [8, 16, 32, 40, 64])
def test_long_calls_of_small_ranks(xk, yk, rank):
    Case([800, 0, 300, 33, 1, 127, 900, 450], [3, 0, 1, -1, 2, 4, 2, 0], rank, 264, 136, xk, yk, before=1, after=3).check()
    Case([1300, 31, 1500], [1, -1, 1], rank, 64, 264, xk, yk, inplace=True, pad=8).check()


FEW = ([0, 1, 8, 9, 17, 0, 3, 2, 0, 1, 1, 7, 0, 5], [3, 0, 1, -1, 2, -1, 4, 2, 0, 0, 1, 1, 2, 2])  # 54 tokens in 14 segments


@pytest.mark.parametrize("xk,yk", list(itertools.product(KINDS, KINDS)))
@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 64, 120, 128])
def test_few_tokens_a_segment(xk, yk, rank):
    Case(*FEW, rank, 520, 392, xk, yk, before=1, after=3).check()
    Case(*FEW, rank, 2560, 2088, xk, yk, base=False).check()
    Case(*FEW, rank, 64, 2560, xk, yk, inplace=True, pad=8).check()


@pytest.mark.parametrize("d_in,d_out", [(8, 8), (8, 16384), (16384, 8), (24, 40), (248, 264), (2552, 2568)])
@pytest.mark.parametrize("lens,of", [([1], [1]), ([8], [0]), ([3, 4], [2, -1]), ([1] * 200, [i % 6 - 1 for i in range(200)])])
def test_few_tokens_widths(d_in, d_out, lens, of):
    Case(lens, of, 16, d_in, d_out).check()
    Case(lens, of, 72, d_in, d_out, qre.BF16, qre.F16).check()


@pytest.mark.parametrize("d_in,d_out", [(8, 8), (8, 2560), (2560, 8), (24, 40), (248, 256), (264, 1032), (2552, 520), (5120, 24),
                                        (16384, 16), (16, 16384)])
def test_widths(d_in, d_out):
    Case(*RAGGED, 16, d_in, d_out).check()
    Case([70], [0], 32, d_in, d_out, qre.F16, qre.BF16).check()
    Case([70, 200], [0, 4], 24, d_in, d_out).check()


@pytest.mark.parametrize("lens,of", [
    ([1], [0]), ([1], [-1]), ([1, 1, 1], [2, 2, 0]), ([16], [1]), ([15, 1], [1, 1]), ([31, 32, 33], [0, 1, 2]), ([64], [4]),
    ([127, 128, 129], [4, 3, 2]), ([1] * 64, [i % 5 for i in range(64)]), ([0] * 300 + [3] + [0] * 300, [0] * 300 + [1] + [-1] * 300),
    ([2048], [3]), ([700, 1, 900, 0, 447], [0, -1, 1, 2, 3]), ([1] * 1000, [(i * 7) % 6 - 1 for i in range(1000)])])
def test_segments(lens, of):
    Case(lens, of, 16, 264, 136).check()
    Case(lens, of, 48, 136, 264, qre.BF16, qre.BF16, before=3, after=2).check()


def test_largest_call():
    lens = np.full(32, 256)
    lens[::2] += 101
    lens[1::2] -= 101
    Case(lens, np.arange(32) % 5, 64, 2560, 2560, qre.BF16, qre.BF16).check()
    Case([8192], [1], 8, 64, 64).check()
    Case([1] * 8192, [i % 5 for i in range(8192)], 8, 64, 64).check()


def test_in_place_no_base_no_scale_strides():
    for kind in KINDS:
        Case(*RAGGED, 16, 264, 136, kind, kind, inplace=True, pad=8, before=4, after=9).check()
        Case(*RAGGED, 16, 264, 136, kind, kind, base=False, pad=16, wpad=8).check()
        Case(*RAGGED, 24, 136, 264, kind, kind, scale=False, pad=8, wpad=16, after=1).check()


def test_no_term_of_an_operand_is_lost():
    """Whole numbers whose sums all fit 24 bits: the result is exact, so a dropped low term of x or of A x shows."""
    T, d_in, d_out, rank = 40, 96, 72, 16
    g = torch.Generator().manual_seed(3)
    x = torch.zeros(T, d_in)
    x[torch.arange(T), torch.randint(0, d_in, (T,), generator=g)] = (torch.randint(0, 1 << 22, (T,), generator=g) * 2 + 1).float()
    a = torch.randint(-1, 2, (1, rank, d_in), generator=g).bfloat16()
    b = torch.zeros(1, d_out, rank)
    b[0, torch.arange(d_out), torch.randint(0, rank, (d_out,), generator=g)] = 1.0
    b = b.bfloat16()
    want = x.double() @ a[0].double().t() @ b[0].double().t()
    assert want.abs().max() < 1 << 24 and (want != 0).any()
    y = torch.empty(T, d_out, device=DEV)
    xd, ad, bd = x.to(DEV), a.to(DEV), b.to(DEV)
    off, of = torch.tensor([0, T], dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = workspace(T)
    qre.strata_moe_adapters(qre.adapters(ad, bd, 1, rank, d_in, d_out), off, of, 1, xd, T, None, y, ws)
    assert torch.equal(y.cpu().double(), want)
    # fp16 activations: 11 bits, two terms
    x16 = (x % 2047).half()
    want = x16.double() @ a[0].double().t() @ b[0].double().t()
    qre.strata_moe_adapters(qre.adapters(ad, bd, 1, rank, d_in, d_out, x_type=qre.F16), off, of, 1, x16.to(DEV), T, None, y, ws)
    assert torch.equal(y.cpu().double(), want)


@pytest.mark.parametrize("off,of", [([0, 5, 3, 8], [0, 1, 2]), ([0, 5, 9, 21], [0, 1, 2]), ([-1, 5, 9, 12], [0, 1, 2]),
                                    ([0, 5, 9, 12], [0, 5, 2]), ([0, 5, 9, 12], [0, 1, -2])])
def test_bad_segments_set_the_status_and_compute_nothing(off, of):
    c = Case([20], [0], 16, 64, 64)
    c.dev_off, c.dev_of = torch.tensor(off, dtype=torch.int32, device=DEV), torch.tensor(of, dtype=torch.int32, device=DEV)
    c.of = np.asarray(of)
    y = c.y.clone()
    c.call()
    assert qre.STATUS[qre.strata_poll_status(c.ws)] == "STRATA_E_CORRUPT"
    assert torch.equal(c.y, y)
    qre.strata_clear_status(c.ws)
    c.dev_off, c.dev_of = torch.tensor([0, 20], dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    c.of = np.zeros(1, np.int32)
    c.check()


def test_repeats_streams_and_graphs():
    c = Case([40, 1, 0, 90], [0, 1, 2, 3], 16, 264, 136, before=2, after=1)
    c.check()
    first = c.y.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.y.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.call()
    side.synchronize()
    assert torch.equal(c.y[2:-1], first[2:-1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call()
        c.call()
    c.x.copy_(rnd(*c.x.shape, seed=77))
    c.y.copy_(first)
    graph.replay()
    torch.cuda.synchronize()
    replayed = c.y.clone()
    c.y.copy_(first)
    c.check()
    assert torch.equal(replayed, c.y)


@pytest.mark.parametrize("T,rank", [(3, 16), (3, 128), (40, 128), (2000, 128)])
def test_no_term_of_an_operand_is_lost_at_any_length(T, rank):
    """As above: one value of x a token, one of B a column, whole numbers."""
    d_in, d_out = 96, 72
    g = torch.Generator().manual_seed(T)
    x = torch.zeros(T, d_in)
    x[torch.arange(T), torch.randint(0, d_in, (T,), generator=g)] = (torch.randint(0, 1 << 22, (T,), generator=g) * 2 + 1).float()
    a = torch.randint(-1, 2, (1, rank, d_in), generator=g).bfloat16()
    b = torch.zeros(1, d_out, rank)
    b[0, torch.arange(d_out), torch.randint(0, rank, (d_out,), generator=g)] = 1.0
    b = b.bfloat16()
    ad, bd = a.to(DEV), b.to(DEV)
    off, of = torch.tensor([0, T], dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = workspace(T)
    for kind, xs in ((qre.F32, x), (qre.F16, (x % 2047).half()), (qre.BF16, (x % 255).bfloat16())):
        y = torch.empty(T, d_out, device=DEV)
        want = xs.double() @ a[0].double().t() @ b[0].double().t()
        qre.strata_moe_adapters(qre.adapters(ad, bd, 1, rank, d_in, d_out, x_type=kind), off, of, 1, xs.to(DEV), T, None, y, ws)
        assert torch.equal(y.cpu().double(), want)


@pytest.mark.parametrize("lens,rank", [([2000], 128), ([1, 2, 3], 16), ([700, 0, 900, 400], 104)])
def test_bad_segments_of_any_length_compute_nothing(lens, rank):
    c = Case(lens, [0] * len(lens), rank, 64, 64)
    good, y = c.dev_off.clone(), c.y.clone()
    for off in ([-1], [c.T + 1], [2 ** 31 - 1], [-2 ** 31]):
        c.dev_off[-1:] = torch.tensor(off, dtype=torch.int32, device=DEV)
        c.call()
        assert qre.STATUS[qre.strata_poll_status(c.ws)] == "STRATA_E_CORRUPT"
        assert torch.equal(c.y, y)
        qre.strata_clear_status(c.ws)
    c.dev_off.copy_(good)
    c.check()


def test_repeats_of_long_segments_in_a_graph():
    c = Case([900, 1, 0, 800], [0, 1, 2, 3], 128, 264, 136, qre.BF16, qre.BF16, before=2, after=1)
    c.check()
    first = c.y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(4):
            c.call()
    for _ in range(3):
        c.y.copy_(first)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.y, first)


def test_calls_on_two_streams_at_once():
    cases = [Case([900, 1, 0, 1100], [0, 1, 2, 3], 128, 520, 392, qre.BF16, qre.BF16, seed=3),
             Case([1500, 700], [4, 4], 104, 264, 520, qre.F32, qre.F32, seed=9),
             Case([1] * 100, [i % 5 for i in range(100)], 16, 520, 392, seed=15),
             Case([40, 3, 90], [1, -1, 1], 24, 264, 136, qre.F16, qre.BF16, seed=21)]
    for c in cases:
        c.check()
    want = [c.y.clone() for c in cases]
    for c in cases:
        c.y.zero_()
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                c.call()
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        assert qre.strata_poll_status(c.ws) == 0 and torch.equal(c.y, w)


@pytest.mark.parametrize("lens,rank", [([2000, 130], 128), ([40, 33], 16), ([1] * 40, 16)])
@pytest.mark.parametrize("kind", KINDS)
def test_bad_numbers_stay_in_their_row(lens, rank, kind):
    c = Case(lens, [i % 5 for i in range(len(lens))], rank, 264, 136, kind, kind, seed=5)
    c.call()
    want = c.y.clone()
    bad = [0, 7, c.T - 1]
    for t, v in zip(bad, (float("nan"), float("inf"), float("-inf"))):
        c.x[t, 3] = v
    c.call()
    torch.cuda.synchronize()
    rest = [t for t in range(c.T) if t not in bad]
    assert torch.equal(c.y[rest], want[rest])
    assert not torch.isfinite(c.y[bad].float()).all(1).any()


# Calls that take tiles of 128 tokens: more than 256K tokens x rank.
@pytest.mark.parametrize("kind", KINDS)
def test_no_term_of_an_operand_is_lost_in_tiles_of_128(kind):
    test_no_term_of_an_operand_is_lost_at_any_length(2500 + kind, 128)


@pytest.mark.parametrize("lens,rank", [([2500], 128), ([1700, 0, 900, 400], 104)])
def test_bad_segments_in_tiles_of_128(lens, rank):
    test_bad_segments_of_any_length_compute_nothing(lens, rank)


def test_tiles_of_128_repeat_and_run_at_once():
    cases = [Case([1400, 1, 0, 1300], [0, 1, 2, 3], 128, 264, 136, qre.BF16, qre.BF16, before=2, after=1),
             Case([2500, 700], [4, 4], 104, 264, 520, qre.F32, qre.F32, seed=9),
             Case([2048, 2900], [1, -1], 72, 520, 264, qre.F16, qre.F16, seed=13, inplace=False),
             Case([1] * 100, [i % 5 for i in range(100)], 16, 520, 392, seed=15)]
    for c in cases:
        c.check()
    want = [c.y.clone() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    graphs = []
    torch.cuda.synchronize()
    for c, s in zip(cases, streams):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            c.call()
            c.call()
    for _ in range(10):
        for c, s, g in zip(cases, streams, graphs):
            with torch.cuda.stream(s):
                c.call()
                g.replay()
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        assert qre.strata_poll_status(c.ws) == 0 and torch.equal(c.y, w)


@pytest.mark.parametrize("kind", KINDS)
def test_bad_numbers_stay_in_their_row_in_tiles_of_128(kind):
    test_bad_numbers_stay_in_their_row([2200, 130], 128, kind)


# 2,500 tokens of rank 128 are 20 tiles and 3,000 in six segments up to 29, so d_in is cut into as many slices as a cluster
# may have CTAs: 8 of 320.
@pytest.mark.parametrize("xk,yk", list(itertools.product(KINDS, KINDS)))
def test_slices_of_d_in_in_tiles_of_128(xk, yk):
    Case([2500], [1], 128, 2560, 264, xk, yk).check()
    for rank in (72, 104):
        Case([1200, 0, 900, 128, 1, 771], [3, 0, 1, -1, 2, 4], rank, 2560, 136, xk, yk, before=1, after=3, pad=8).check()


@pytest.mark.parametrize("d_in", [512, 520, 1032, 1096, 1544, 2048, 4104])
def test_slices_of_any_width_in_tiles_of_128(d_in):
    Case([2500], [1], 128, d_in, 72).check()
    Case([2500], [1], 128, d_in, 72, qre.BF16, qre.BF16).check()


@pytest.mark.parametrize("d_in", [2056, 2120, 2568])
@pytest.mark.parametrize("kind", KINDS)
def test_widths_that_eight_slices_do_not_divide(d_in, kind):
    """Slices are whole blocks of 64 columns: 2,056 and 2,120 columns are 7 slices of 320, 2,568 are 7 of 384."""
    Case([2500], [1], 128, d_in, 72, kind, kind).check()
    Case([1200, 0, 900, 128, 1, 771], [3, 0, 1, -1, 2, 4], 104, d_in, 136, kind, kind, before=1, after=3, pad=8).check()


def check_rows_without_an_adapter(lens, of, rank, kind, base=True):
    c = Case(lens, of, rank, 264, 136, kind, kind, base=base)
    if base:
        c.base[:, ::3] = -0.0
        c.base[:, 1::7] *= torch.finfo(c.base.dtype).tiny  # some below the normal numbers
        c.base[:, 5] = float("inf")
    c.call()
    assert qre.strata_poll_status(c.ws) == 0
    bits = torch.int32 if kind == qre.F32 else torch.int16
    for i, ad in enumerate(of):
        if ad < 0:
            s = slice(c.off[i], c.off[i + 1])
            want = c.base[s] if base else torch.zeros_like(c.y[s])
            assert torch.equal(c.y[s].contiguous().view(bits), want.contiguous().view(bits))


@pytest.mark.parametrize("lens,of", [([3, 1, 5], [-1, 0, -1]), ([200, 1100, 300], [-1, 2, -1]), ([1500, 2600, 31], [-1, 2, -1])])
@pytest.mark.parametrize("kind", KINDS)
def test_rows_without_an_adapter_keep_base_bit_for_bit(lens, of, kind):
    for rank in (16, 32):
        check_rows_without_an_adapter(lens, of, rank, kind)
        check_rows_without_an_adapter(lens, of, rank, kind, base=False)


@pytest.mark.parametrize("kind", KINDS)
def test_rows_without_an_adapter_keep_base_in_tiles_of_128(kind):
    check_rows_without_an_adapter([300, 2500, 130], [-1, 2, -1], 128, kind)
    check_rows_without_an_adapter([300, 2500, 130], [-1, 2, -1], 128, kind, base=False)


def check_column_ranges(T, rank):
    n = 136
    a, b = rnd(2, rank, n, seed=31, std=n ** -0.5, kind=qre.BF16), rnd(2, n, rank, seed=32, std=rank ** -0.5, kind=qre.BF16)
    off, of = torch.tensor([0, T // 2, T], dtype=torch.int32, device=DEV), torch.tensor([1, -1], dtype=torch.int32, device=DEV)
    ws = workspace(T)
    for kind in KINDS:
        buf = rnd(T, 3 * n, seed=33, kind=kind)
        x, base, y = buf[:, :n], buf[:, n:2 * n], buf[:, 2 * n:]
        x0, base0 = x.contiguous(), base.contiguous()
        want = torch.empty_like(x0)
        qre.strata_moe_adapters(qre.adapters(a, b, 2, rank, n, n, x_type=kind, y_type=kind), off, of, 2, x0, T, base0, want, ws)
        d = qre.adapters(a, b, 2, rank, n, n, x_type=kind, y_type=kind, x_stride=3 * n, base_stride=3 * n, y_stride=3 * n)
        qre.strata_moe_adapters(d, off, of, 2, x.data_ptr(), T, base.data_ptr(), y.data_ptr(), ws)
        assert qre.strata_poll_status(ws) == 0
        assert torch.equal(y, want) and torch.equal(x, x0) and torch.equal(base, base0)


@pytest.mark.parametrize("T,rank", [(1, 16), (40, 32), (1500, 16)])
def test_column_ranges_of_one_buffer(T, rank):
    check_column_ranges(T, rank)


def test_column_ranges_of_one_buffer_in_tiles_of_128():
    check_column_ranges(2500, 128)


FIRST_RANK = """
import hashlib, sys, torch, quantized_routed_expert_top10_gb300 as qre
out = {}
for rank in map(int, sys.argv[1:]):
    for lens in ([9] * 20, [40] * 5, [100] * 40):
        T, n = sum(lens), 1032
        g = torch.Generator("cuda").manual_seed(rank)
        a, b = (torch.randn(5, rank, n, generator=g, device="cuda").bfloat16() for _ in range(2))
        x = torch.randn(T, n, generator=g, device="cuda")
        off = torch.tensor([0] + lens, device="cuda").cumsum(0).int()
        of = (torch.arange(len(lens), device="cuda") % 5).int()
        ws = torch.empty(qre.strata_moe_workspace_bytes(T), dtype=torch.uint8, device="cuda")
        qre.strata_moe_workspace_init(ws)
        y = torch.empty(T, n, device="cuda")
        qre.strata_moe_adapters(qre.adapters(a, b, 5, rank, n, n), off, of, len(lens), x, T, None, y, ws)
        assert qre.strata_poll_status(ws) == 0
        out[rank, T] = hashlib.sha256(y.cpu().numpy().tobytes()).hexdigest()
print(sorted(out.items()))
"""


def test_the_rank_of_a_process_first_call_changes_no_bits():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    got = set()
    for ranks in (("40", "128", "64"), ("128", "64", "40")):
        r = subprocess.run([sys.executable, "-c", FIRST_RANK, *ranks], cwd=root, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stdout + r.stderr
        got.add(r.stdout)
    assert len(got) == 1 and "(40, 180)" in got.pop()
