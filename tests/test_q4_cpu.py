"""4-bit weights without a GPU: the packed layout against its description, and every refusal of the host-side checks of the packers,
strata_moe_linear and strata_moe_q4_experts (which come before anything is enqueued)."""
import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

import q4_reference as q4ref
import quantized_routed_expert_top10_gb300 as qre
from conftest import ROOT

HEADER = os.path.join(ROOT, "include", "strata_moe_ops.h")
A = 1 << 20                      # an aligned address; nothing of it is read
X, Y, Z, V, W = (A + (i << 40) for i in range(5))  # far apart: no overlap
INVAL, ALIGN, WORKSPACE = -1, -2, -6


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(qre.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return qre.lib()


def with_(d, **changes):
    c = type(d).from_buffer_copy(d)
    for k, v in changes.items():
        setattr(c, k, v)
    return c


def test_constants_match_the_header():
    c = dict(re.findall(r"#define (STRATA_[A-Z0-9_]+) (\d+)", open(HEADER).read()))
    for name in ("W_Q4", "W_BF16", "Q4_ROWS_MAX", "Q4_COLUMNS_MAX", "Q4_EXPERTS_T_MAX", "Q4_EXPERTS_DIM_MAX", "Q4_EXPERTS_E_MAX",
                 "Q4_EXPERTS_K_MAX"):
        assert int(c["STRATA_" + name]) == getattr(qre, name), name


def test_descriptor_layouts_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if not cc:
        pytest.skip("no C compiler")
    lines = ["#include <stdio.h>", '#include "strata_moe_ops.h"', "int main(void) {"]
    want = []
    for t in (qre.strata_q4_t, qre.strata_linear_t, qre.strata_q4_experts_t):
        lines.append(f'  printf("%zu\\n", sizeof({t.__name__}));')
        want.append(ctypes.sizeof(t))
        for f, _ in t._fields_:
            lines.append(f'  printf("%zu\\n", offsetof({t.__name__}, {f}));')
            want.append(getattr(t, f).offset)
    (tmp_path / "l.c").write_text("\n".join(lines + ["  return 0;", "}"]))
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), "-o", str(tmp_path / "l"), str(tmp_path / "l.c")], check=True)
    got = subprocess.run([str(tmp_path / "l")], check=True, capture_output=True, text=True).stdout.split()
    assert [int(v) for v in got] == want


@pytest.mark.parametrize("group,d_in", [(32, 32), (32, 160), (32, 224), (32, 256), (64, 64), (64, 192), (64, 320), (128, 128), (128, 384)])
@pytest.mark.parametrize("zeros", [False, True])
def test_packed_layout(lib, group, d_in, zeros):
    for n_out, paired in ((1, False), (16, False), (37, False), (16, True), (48, True)):
        m = q4ref.Matrices(2, n_out, d_in, group, zeros, qre.F16 if zeros else qre.BF16, paired, seed=d_in + n_out)
        got = m.packed_host().numpy()
        for i in range(2):
            want = q4ref.packed_from_description(m, i)
            assert got.shape[1] == want.size and want.size % 32 == 0
            np.testing.assert_array_equal(got[i], want)


def test_zero_points_above_four_bits_are_cut(lib):
    m = q4ref.Matrices(1, 16, 128, 32, True)
    want = m.packed_host()
    m.zeros = m.zeros | 0x50
    assert torch.equal(m.packed_host(), want)


GOOD = qre.q4(32, 256, 64)
BAD_FORMATS = [dict(n_out=0), dict(n_out=-1), dict(n_out=qre.Q4_ROWS_MAX + 1), dict(d_in=0), dict(d_in=32), dict(d_in=96),
               dict(d_in=qre.Q4_COLUMNS_MAX + 64), dict(group=0), dict(group=16), dict(group=256), dict(scale_type=qre.F32),
               dict(scale_type=3), dict(zeros=2), dict(zeros=-1), dict(paired=2), dict(paired=1, n_out=24)]


def test_format_refusals(lib):
    f, h = lib.strata_pack_q4_device, lib.strata_pack_q4
    assert lib.strata_q4_bytes(None) == 0
    assert lib.strata_q4_bytes(ctypes.byref(GOOD)) == 2 * (2 * (1024 + 64))
    for c in BAD_FORMATS:
        bad = with_(GOOD, **c)
        assert lib.strata_q4_bytes(ctypes.byref(bad)) == 0, c
        assert f(ctypes.byref(bad), X, Y, Z if bad.zeros else None, V, 1, None) == INVAL, c
        assert h(ctypes.byref(bad), X, Y, Z if bad.zeros else None, V, 1) == INVAL, c
    for zeros, q in ((None, GOOD), (Z, with_(GOOD, zeros=1))):
        ok = [ctypes.byref(q), X, Y, zeros, V, 0, None]
        assert f(*ok) == 0 and h(*ok[:-1]) == 0
        for i in (0, 1, 2, 4):
            args = list(ok)
            args[i] = None
            assert f(*args) == INVAL and h(*args[:-1]) == INVAL
        assert f(ctypes.byref(q), X, Y, Z if zeros is None else None, V, 0, None) == INVAL
        assert f(ctypes.byref(q), X, Y, zeros, V, -1, None) == INVAL
        assert f(ctypes.byref(q), X, Y, zeros, V, 65537, None) == INVAL
        assert f(ctypes.byref(q), X, Y + 1, zeros, V, 0, None) == ALIGN
        assert f(ctypes.byref(q), X, Y, zeros, V + 8, 0, None) == ALIGN


def test_linear_refusals(lib):
    f = lib.strata_moe_linear

    def call(d, x=X, T=0, bias=None, y=Y):
        return f(ctypes.byref(d), x, T, bias, y, None)

    d, b = qre.linear_q4(GOOD, W), qre.linear_bf16(W, 24, 40)
    assert f(None, X, 0, None, Y, None) == INVAL
    for d0 in (d, b):
        assert call(d0) == 0 and call(d0, bias=Z) == 0
        assert call(d0, x=None) == INVAL and call(d0, y=None) == INVAL and call(with_(d0, w=None)) == INVAL
        assert call(d0, T=-1) == INVAL and call(d0, T=qre.T_MAX + 1) == INVAL
        for k in ("x_type", "y_type", "weight"):
            assert call(with_(d0, **{k: 3})) == INVAL and call(with_(d0, **{k: -1})) == INVAL
        assert call(with_(d0, reserved=1)) == INVAL
        assert call(with_(d0, x_stride=d0.q4.d_in - 8)) == INVAL and call(with_(d0, y_stride=d0.q4.n_out - 1)) == INVAL
        assert call(with_(d0, x_stride=1 << 41)) == INVAL and call(with_(d0, y_stride=1 << 41)) == INVAL
        assert call(with_(d0, x_stride=d0.q4.d_in + 4)) == ALIGN
        assert call(with_(d0, y_stride=d0.q4.n_out + 1)) == 0
        assert call(with_(d0, w=W + 8)) == ALIGN and call(d0, x=X + 8) == ALIGN
        assert call(d0, y=Y + 2) == ALIGN and call(with_(d0, y_type=qre.BF16), y=Y + 2) == 0
        assert call(d0, bias=Z + 2) == ALIGN
        assert call(d0, T=2, bias=Y + 64) == INVAL  # bias in y
        # y in x, and x in y
        assert call(d0, T=2, y=X + 16) == INVAL and call(d0, T=2, y=X - 16) == INVAL
    for c in BAD_FORMATS:
        assert call(with_(d, q4=with_(GOOD, **c))) == INVAL, c
    assert call(with_(d, q4=with_(GOOD, paired=1))) == INVAL
    assert call(with_(d, w_stride=256)) == INVAL
    for c in (dict(n_out=0), dict(n_out=qre.Q4_ROWS_MAX + 1), dict(d_in=0), dict(d_in=36), dict(d_in=qre.Q4_COLUMNS_MAX + 8),
              dict(group=64), dict(scale_type=1), dict(zeros=1), dict(paired=1)):
        assert call(with_(b, q4=with_(b.q4, **c))) == INVAL, c
    assert call(with_(b, w_stride=32)) == INVAL and call(with_(b, w_stride=44)) == ALIGN and call(with_(b, w_stride=48)) == 0


def test_experts_refusals(lib):
    f, size = lib.strata_moe_q4_experts, lib.strata_moe_q4_experts_workspace_bytes
    gu, dn = qre.q4(2 * 96, 128, 32, paired=True), qre.q4(128, 96, 32)
    d = qre.q4_experts(gu, W, dn, W + (1 << 30), 8, 4)
    WS = A + (7 << 40)

    def call(d, ids=Y, weights=Z, x=X, T=0, out=V, ws=WS, ws_bytes=1 << 30):
        return f(ctypes.byref(d), ids, weights, x, T, out, ws, ws_bytes, None)

    assert call(d) == 0
    assert f(None, Y, Z, X, 0, V, WS, 1 << 30, None) == INVAL and size(None, 1) == 0
    for k in ("ids", "weights", "x", "out", "ws"):
        assert call(d, **{k: None}) == INVAL, k
    assert call(with_(d, gate_up=None)) == INVAL and call(with_(d, down=None)) == INVAL
    for T in (-1, qre.Q4_EXPERTS_T_MAX + 1):
        assert call(d, T=T) == INVAL and size(ctypes.byref(d), T) == 0
    wide = qre.Q4_EXPERTS_DIM_MAX + 32
    for c in (dict(n_expert=0), dict(n_expert=qre.Q4_EXPERTS_E_MAX + 1), dict(top_k=0), dict(top_k=qre.Q4_EXPERTS_K_MAX + 1),
              dict(x_type=3), dict(out_type=-1), dict(x_stride=120), dict(out_stride=120), dict(x_stride=1 << 41),
              dict(gate_up_stride=qre.strata_q4_bytes(gu) - 16), dict(down_stride=qre.strata_q4_bytes(dn) - 16),
              dict(gate_up_q4=with_(gu, paired=0)), dict(down_q4=with_(dn, paired=1)), dict(down_q4=with_(dn, d_in=128)),
              dict(down_q4=with_(dn, n_out=256)), dict(gate_up_q4=with_(gu, d_in=256)), dict(gate_up_q4=with_(gu, group=48)),
              dict(down_q4=with_(dn, group=64)), dict(down_q4=with_(dn, scale_type=qre.F16)), dict(down_q4=with_(dn, zeros=1)),
              dict(gate_up_q4=with_(gu, group=64)),
              dict(gate_up_q4=with_(gu, d_in=wide), down_q4=with_(dn, n_out=wide), x_stride=wide, out_stride=wide,
                   gate_up_stride=1 << 25, down_stride=1 << 25),
              dict(gate_up_q4=with_(gu, n_out=2 * wide), down_q4=with_(dn, d_in=wide), gate_up_stride=1 << 25,
                   down_stride=1 << 25)):
        bad = with_(d, **c)
        assert call(bad) == INVAL, c
        assert size(ctypes.byref(bad), 1) == 0, c
    for c in (dict(gate_up=W + 8), dict(down=W + 8), dict(gate_up_stride=d.gate_up_stride + 8), dict(down_stride=d.down_stride + 8),
              dict(x_stride=132), dict(out_stride=132)):
        assert call(with_(d, **c)) == ALIGN, c
    for k, a in (("ids", Y + 2), ("weights", Z + 2), ("x", X + 8), ("out", V + 8), ("ws", WS + 128)):
        assert call(d, **{k: a}) == ALIGN, k
    for T in (0, 1, 64):
        need = size(ctypes.byref(d), T)
        assert need > 0 and call(d, T=T, ws_bytes=need - 1) == WORKSPACE
    assert call(d, T=2, out=X + 16) == INVAL and call(d, T=2, ids=V + 64) == INVAL and call(d, T=2, weights=V + 128 * 4) == INVAL
