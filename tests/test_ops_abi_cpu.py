"""The operators of strata_moe_ops.h without a GPU: exported symbols, descriptor layouts, and every refusal of the
host-side checks (which come before anything is enqueued)."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

import quantized_routed_expert_top10_gb300 as qre
from conftest import ROOT

HEADER = os.path.join(ROOT, "include", "strata_moe_ops.h")
A = 1 << 20                      # an aligned address; nothing of it is read
X, Y, Z, V = (A + (i << 34) for i in range(4))  # far apart: no overlap
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


def test_exports_every_declared_symbol(lib):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(strata_[a-z0-9_]+)\s*\(", src)))
    assert names == sorted(qre.OPS_EXPORTS)
    for n in names:
        assert hasattr(lib, n), n


def test_constants_match_the_header():
    c = dict(re.findall(r"#define (STRATA_[A-Z0-9_]+) (\d+)", open(HEADER).read()))
    for name, value in (("F32", qre.F32), ("BF16", qre.BF16), ("F16", qre.F16), ("SCORE_SOFTMAX", qre.SCORE_SOFTMAX),
                        ("SCORE_SIGMOID", qre.SCORE_SIGMOID), ("SELECT_K_MAX", qre.SELECT_K_MAX),
                        ("SELECT_GROUP_MAX", qre.SELECT_GROUP_MAX), ("NORM_N_MAX", qre.NORM_N_MAX),
                        ("NORM_PART_MAX", qre.NORM_PART_MAX), ("POST_NORM", qre.POST_NORM),
                        ("TOKEN_SIGMOID", qre.TOKEN_SIGMOID), ("ADAPTER_RANK_MAX", qre.ADAPTER_RANK_MAX),
                        ("ADAPTER_DIM_MAX", qre.ADAPTER_DIM_MAX), ("ADAPTER_COUNT_MAX", qre.ADAPTER_COUNT_MAX)):
        assert int(c["STRATA_" + name]) == value, name


def test_descriptor_layouts_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if not cc:
        pytest.skip("no C compiler")
    lines = ["#include <stdio.h>", '#include "strata_moe_ops.h"', "int main(void) {"]
    want = []
    for t in (qre.strata_select_t, qre.strata_norm_t, qre.strata_combine_norm_t, qre.strata_adapters_t):
        lines.append(f'  printf("%zu\\n", sizeof({t.__name__}));')
        want.append(ctypes.sizeof(t))
        for f, _ in t._fields_:
            lines.append(f'  printf("%zu\\n", offsetof({t.__name__}, {f}));')
            want.append(getattr(t, f).offset)
    (tmp_path / "l.c").write_text("\n".join(lines + ["  return 0;", "}"]))
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), "-o", str(tmp_path / "l"), str(tmp_path / "l.c")], check=True)
    got = subprocess.run([str(tmp_path / "l")], check=True, capture_output=True, text=True).stdout.split()
    assert [int(v) for v in got] == want


def test_select_refusals(lib):
    f = lib.strata_moe_select
    d = qre.select(512, 10, qre.SCORE_SIGMOID, n_group=16, top_group=4, group_sum=2)

    def call(d=d, logits=X, T=4, bias=None, ids=Y, weights=Z):
        return f(ctypes.byref(d), logits, T, bias, ids, weights, None)

    assert f(None, X, 4, None, Y, Z, None) == INVAL
    for k in ("logits", "ids", "weights"):
        assert call(**{k: None}) == INVAL
    assert call(T=-1) == INVAL and call(T=8193) == INVAL
    for field, values in (("n_expert", (0, -16, 513, 528, 500)), ("n_group", (0, 33, 64, 7)), ("top_group", (0, 17)),
                          ("group_sum", (0, 3)), ("top_k", (0, -1, 33)), ("score", (-1, 2)), ("renorm", (2, -1)),
                          ("scale", (float("nan"), float("inf"))), ("logits_type", (-1, 3)), ("reserved", (1,)),
                          ("logits_stride", (511, -1, 1 << 41))):
        for v in values:
            assert call(with_(d, **{field: v})) == INVAL, (field, v)
    # more experts than the kept groups hold
    assert call(qre.select(64, 9, n_group=8, top_group=1)) == INVAL
    assert call(logits=X + 2) == ALIGN and call(ids=Y + 2) == ALIGN and call(weights=Z + 1) == ALIGN and call(bias=V + 2) == ALIGN
    assert call(with_(d, logits_type=qre.BF16), logits=X + 1) == ALIGN
    # outputs over the logits or each other
    assert call(ids=X + 64) == INVAL and call(weights=X) == INVAL and call(weights=Y + 4) == INVAL
    assert call(T=0) == 0


def test_norm_refusals(lib):
    d = qre.norm(2560)

    def call(d=d, x=X, T=4, gain=None, out=Y):
        return lib.strata_moe_norm(ctypes.byref(d), x, T, gain, out, None)

    assert lib.strata_moe_norm(None, X, 4, None, Y, None) == INVAL
    assert call(x=None) == INVAL and call(out=None) == INVAL and call(T=-1) == INVAL and call(T=8193) == INVAL
    for field, values in (("n", (0, -1, 16385)), ("eps", (-1e-6, float("nan"), float("inf"))), ("x_type", (3, -1)),
                          ("out_type", (3, -1)), ("x_stride", (2559, 1 << 41)), ("out_stride", (0, 2559))):
        for v in values:
            assert call(with_(d, **{field: v})) == INVAL, (field, v)
    assert call(x=X + 2) == ALIGN and call(out=Y + 2) == ALIGN and call(gain=Z + 2) == ALIGN
    # partly overlapping rows, and the same address with another type or stride
    assert call(out=X + 4) == INVAL and call(qre.norm(2560, out_type=qre.BF16), out=X) == INVAL
    assert call(qre.norm(2560, out_stride=2568), out=X) == INVAL
    assert call(T=0) == 0


def test_combine_norm_refusals(lib):
    d = qre.combine_norm()

    def call(d=d, parts=X, pw=None, x=Y, T=4, post=None, channel=None, token=None, pre=None, out=Z, next=V):
        return lib.strata_moe_combine_norm(ctypes.byref(d), parts, pw, x, T, post, channel, token, pre, out, next, None)

    assert lib.strata_moe_combine_norm(None, X, None, Y, 4, None, None, None, None, Z, V, None) == INVAL
    assert call(parts=None) == INVAL and call(out=None, next=None) == INVAL and call(T=-1) == INVAL and call(T=8193) == INVAL
    for field, values in (("n", (0, 16385)), ("n_part", (0, 33)), ("flags", (4, 8)), ("eps", (-1.0, float("nan"))),
                          ("residual_scale", (float("inf"),)), ("block_scale", (float("nan"),)), ("part_type", (3,)),
                          ("x_type", (-1,)), ("next_type", (3,)), ("reserved", (1,)), ("part_stride", (2559, 1 << 41)),
                          ("token_stride", (25599, 1 << 41)), ("x_stride", (2559,)), ("out_stride", (2559,)),
                          ("next_stride", (2559,))):
        for v in values:
            assert call(with_(d, **{field: v})) == INVAL, (field, v)
    # what nothing would apply
    assert call(qre.combine_norm(post_norm=False), post=A) == INVAL
    assert call(qre.combine_norm(token_sigmoid=True)) == INVAL
    assert call(pre=A, next=None) == INVAL
    assert call(parts=X + 2) == ALIGN and call(x=Y + 2) == ALIGN and call(out=Z + 2) == ALIGN and call(next=V + 2) == ALIGN
    for k in ("pw", "post", "channel", "token", "pre"):
        assert call(**{k: A + 2}) == ALIGN, k
    # overlaps: parts with an output, out with next, x with an output in part
    assert call(out=X) == INVAL and call(next=X + 4096) == INVAL and call(next=Z) == INVAL
    assert call(out=Y + 4) == INVAL and call(next=Y + 10240) == INVAL
    assert call(T=0) == 0


def test_adapters_refusals(lib):
    d = qre.adapters(A, A, 4, 16)
    ws = A
    need = qre.strata_moe_workspace_bytes(4)

    def call(d=d, off=A, of=A, n_seg=2, x=X, T=4, base=Y, y=Z, ws=ws, ws_bytes=need):
        return lib.strata_moe_adapters(ctypes.byref(d), off, of, n_seg, x, T, base, y, ws, ws_bytes, None)

    assert lib.strata_moe_adapters(None, A, A, 2, X, 4, Y, Z, ws, need, None) == INVAL
    for k in ("off", "of", "x", "y", "ws"):
        assert call(**{k: None}) == INVAL, k
    assert call(T=-1) == INVAL and call(T=8193) == INVAL and call(n_seg=-1) == INVAL and call(n_seg=8193) == INVAL
    for field, values in (("a", (None,)), ("b", (None,)), ("n_adapter", (0, 65537)), ("rank", (0, 7, 12, 136)),
                          ("d_in", (0, 4, 12, 16392)), ("d_out", (0, 4, 12, 16392)), ("x_type", (3,)), ("y_type", (-1,)),
                          ("a_stride", (16 * 2560 - 8, 1 << 41)), ("b_stride", (16 * 2560 - 8,)), ("x_stride", (2552,)),
                          ("base_stride", (2552,)), ("y_stride", (2552,))):
        for v in values:
            assert call(with_(d, **{field: v})) == INVAL, (field, v)
    for field in ("a_stride", "b_stride", "x_stride", "base_stride", "y_stride"):
        assert call(with_(d, **{field: getattr(d, field) + 4})) == ALIGN, field
    assert call(with_(d, base_stride=7), base=None, T=0) == 0  # not looked at without a base
    for field in ("a", "b"):
        assert call(with_(d, **{field: A + 8})) == ALIGN, field
    assert call(with_(d, scale=A + 2)) == ALIGN
    assert call(x=X + 8) == ALIGN and call(base=Y + 8) == ALIGN and call(y=Z + 8) == ALIGN
    assert call(off=A + 2) == ALIGN and call(of=A + 2) == ALIGN and call(ws=A + 128) == ALIGN
    assert call(ws_bytes=need - 1) == WORKSPACE
    # y over x, y over a part of base, y as base with another stride
    assert call(y=X) == INVAL and call(y=Y + 10240) == INVAL and call(with_(d, y_stride=2568), y=Y) == INVAL
    assert call(T=0) == 0 and call(n_seg=0) == 0


def test_binding_raises_with_the_status():
    with pytest.raises(qre.StrataError) as e:
        qre.strata_moe_select(qre.select(512, 33), X, 1, None, Y, Z, stream=0)
    assert e.value.status == INVAL
    with pytest.raises(qre.StrataError):
        qre.strata_moe_norm(qre.norm(0), X, 1, None, Y, stream=0)
    with pytest.raises(qre.StrataError):
        qre.strata_moe_combine_norm(qre.combine_norm(n_part=0), X, None, Y, 1, None, None, None, None, Z, V, stream=0)
    with pytest.raises(qre.StrataError):
        qre.strata_moe_adapters(qre.adapters(A, A, 1, 4), A, A, 1, X, 1, Y, Z, A, ws_bytes=1 << 40, stream=0)


def test_rows_that_meet_are_refused_whatever_their_strides(lib):
    """Rows that share an element, of operands whose rows lie between each other's."""
    n, T, s = 64, 9, 4 * 160  # rows of 64 fp32, 160 apart

    def norm(x, out, xs=160, os=160, xt=qre.F32, ot=qre.F32, T=T):
        return lib.strata_moe_norm(ctypes.byref(qre.norm(n, x_type=xt, out_type=ot, x_stride=xs, out_stride=os)), x, T, None, out, None)

    for shift in (4, 4 * 63, s - 4 * 63, s + 4 * 63, 8 * s, 8 * s - 4 * 63, 8 * s + 4 * 63):
        assert norm(X, X + shift) == INVAL and norm(X + shift, X) == INVAL, shift
    # the rows of one meet those of the other once, at the last row, by their strides
    assert norm(X, X + 256, os=161 - 8) == INVAL and norm(X + 256, X, xs=161 - 8) == INVAL
    assert norm(X, X + 2 * 512, xs=512, os=96, T=200) == INVAL
    # bytes count, not elements
    assert norm(X, X + 128, ot=qre.BF16, os=320) == INVAL
    # one of the parts, in the middle of a token's
    d = qre.combine_norm(n, 3, part_stride=160, token_stride=640, out_stride=640, next_stride=640)
    for at in (0, 160, 320, 640 * 8 + 320, 97, 383):
        assert lib.strata_moe_combine_norm(ctypes.byref(d), X, None, None, T, None, None, None, None, X + 4 * at, None, None) == INVAL, at
        assert lib.strata_moe_combine_norm(ctypes.byref(d), X, None, None, T, None, None, None, None, None, X + 4 * at, None) == INVAL, at
    need = qre.strata_moe_workspace_bytes(T)
    a = qre.adapters(A, A, 4, 16, n, n, x_stride=160, y_stride=160, base_stride=160)
    for shift in (32, 4 * 56, s - 4 * 56, 8 * s + 32):
        assert lib.strata_moe_adapters(ctypes.byref(a), A, A, 2, X, T, None, X + shift, A, need, None) == INVAL, shift
        assert lib.strata_moe_adapters(ctypes.byref(a), A, A, 2, Y, T, X, X + shift, A, need, None) == INVAL, shift
    sel = qre.select(n, 10, logits_stride=160)
    assert lib.strata_moe_select(ctypes.byref(sel), X, 40, None, X + 4 * 64, Z, None) == INVAL
