"""strata_moe_linear with bf16 weights of many rows and activations that do not all lie in shared memory at once (panels of columns, one or several
warps to 16 rows), against the formula in 64 bits and against itself."""
import pytest
import torch

import ops_reference as ref
import quantized_routed_expert_top10_gb300 as qre

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def check(T, xk, d_in, n_out, pad=0):
    g = torch.Generator(DEV).manual_seed(T + d_in + n_out)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    w = torch.empty(n_out, d_in + pad, dtype=torch.bfloat16, device=DEV)
    for lo in range(0, n_out, 16384):  # in pieces: no fp32 copy of a whole vocabulary
        w[lo:lo + 16384] = (rnd(min(16384, n_out - lo), d_in + pad) * d_in ** -0.5).bfloat16()
    x, bias = rnd(T, d_in + pad).to(ref.TORCH[xk]), rnd(n_out)
    d = qre.linear_bf16(w, n_out, d_in, xk, qre.F32, d_in + pad, d_in + pad)
    y, again = torch.full((T + 1, n_out), 7.0, device=DEV), torch.empty(T, n_out, device=DEV)
    qre.strata_moe_linear(d, x, T, bias, y)
    for _ in range(3):
        qre.strata_moe_linear(d, x, T, bias, again)
        assert torch.equal(again, y[:T])
    assert (y[T] == 7.0).all()  # nothing behind the last row
    x64 = x[:, :d_in].double()
    for lo in range(0, n_out, 16384):
        w64 = w[lo:lo + 16384, :d_in].double()
        b64 = bias[lo:lo + 16384].double()
        want = x64 @ w64.T + b64
        # products of terms are exact; an MMA's 16 products are two additions of up to 2 u to its sum, a warp's MMAs may all follow one another, then up to
        # 16 warps' sums of 3 terms; then the bias
        err = (2 * -(-d_in // 16) + 48) * 2 * ref.U * (x64.abs() @ w64.abs().T) + ref.U * want.abs()
        ref.check(y[:T, lo:lo + 16384], want.cpu().numpy(), err.cpu().numpy(), qre.F32, f"{T} x {d_in} -> {n_out}, rows from {lo}")


@pytest.mark.parametrize("T,xk,d_in,n_out", [
    (64, qre.BF16, 2560, 10240), (49, qre.BF16, 2560, 10240), (32, qre.BF16, 2560, 32000), (24, qre.BF16, 2560, 32000), (25, qre.BF16, 2560, 131072),
    (64, qre.BF16, 2560, 12800), (16, qre.BF16, 4096, 32000), (145, qre.BF16, 4096, 4096), (241, qre.BF16, 2560, 2560), (8, qre.BF16, 8192, 131072),
    (10, qre.F16, 2560, 32768), (8, qre.F16, 4096, 32000), (7, qre.F32, 2560, 32768), (2, qre.BF16, 32704, 2432),
    (2048, qre.BF16, 2560, 512), (1200, qre.BF16, 2560, 512)])
def test_many_rows_in_panels(T, xk, d_in, n_out):
    check(T, xk, d_in, n_out)


@pytest.mark.parametrize("T,xk,d_in,n_out", [(64, qre.BF16, 2568, 10241), (33, qre.BF16, 2600, 31999), (25, qre.F16, 2616, 20001), (9, qre.F32, 2552, 20001),
                                             (17, qre.BF16, 4024, 32001), (73, qre.BF16, 2504, 5001), (8, qre.F32, 32696, 517)])
def test_odd_sizes_in_panels(T, xk, d_in, n_out):
    """Columns off a multiple of 128, 64 and 32, last blocks of few tokens, a last unit of one row, padded rows."""
    check(T, xk, d_in, n_out, pad=8)


def test_each_column_in_its_place():
    """One column of each token's x is not 0: every weight by itself, across the panels' ends.  bf16 by bf16 is exact, sums with zeros too."""
    T, d_in, n_out = 64, 2560, 10240
    w = (torch.randn(n_out, d_in, generator=torch.Generator(DEV).manual_seed(1), device=DEV)).bfloat16()
    d = qre.linear_bf16(w, n_out, d_in, qre.BF16, qre.F32)
    y = torch.empty(T, n_out, device=DEV)
    for lo in range(0, d_in, T):
        x = torch.zeros(T, d_in, dtype=torch.bfloat16, device=DEV)
        x[torch.arange(T), lo + torch.arange(T)] = 1.0
        qre.strata_moe_linear(d, x, T, None, y)
        assert torch.equal(y, w[:, lo:lo + T].t().float()), lo


def test_panels_in_a_graph_and_beside_others():
    T, d_in, n_out = 64, 2560, 10240
    g = torch.Generator(DEV).manual_seed(2)
    w = (torch.randn(n_out, d_in, generator=g, device=DEV) * d_in ** -0.5).bfloat16()
    d = qre.linear_bf16(w, n_out, d_in, qre.BF16, qre.BF16)
    x = [torch.randn(T, d_in, generator=g, device=DEV).bfloat16() for _ in range(2)]
    want, got = ([torch.empty(T, n_out, dtype=torch.bfloat16, device=DEV) for _ in x] for _ in range(2))
    for a, b in zip(x, want):
        qre.strata_moe_linear(d, a, T, None, b)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in x]
    for _ in range(10):
        for s, a, b in zip(streams, x, got):
            qre.strata_moe_linear(d, a, T, None, b, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qre.strata_moe_linear(d, x[0], T, None, got[0])
    got[0].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0])
