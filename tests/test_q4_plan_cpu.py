"""What a launch of strata_moe_linear lays out in shared memory, walked without a GPU over token counts, types and widths: activations stay in their
rows and in the memory that was asked for, and panels begin and end where the kernel's warps and half warps expect it."""
import ctypes
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

SMEM_MAX = 227 * 1024 - 256
CHUNK = 128  # columns that a half warp lays out at once

# kernels: (tiles, warps, depth, slot, columns, slabs), one tile and up to three
BF16 = ((1, 8, 6, 2048, 64, 1), (3, 16, 3, 2048, 64, 1))


def q4_kernels(meta):
    return ((1, 8, 6, 1024 + meta, 128, 1), (1, 8, 4, 2 * (1024 + meta), 128, 2), (3, 16, 3, 1024 + meta, 128, 1))


class Kernel(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("tiles", "warps", "depth", "slot", "columns", "slabs")]


class Plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("tokens", "part_cols", "log_split", "panel", "row_stride", "scale_stride", "grid_x", "grid_y")] + [
        ("pair", ctypes.c_bool), ("bytes", ctypes.c_size_t)]


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no C++ compiler")
    at = tmp_path_factory.mktemp("plan")
    (at / "p.cc").write_text('#include "q4_sizes.h"\n'
                             'extern "C" void plan(const strata::q4::LinearKernel* k, int T, int columns, int rows, int terms, int sms,\n'
                             '                     strata::q4::LinearPlan* p) { *p = strata::q4::linear_plan(*k, T, columns, rows, terms, sms); }\n')
    csrc = os.path.join(ROOT, "quantized_routed_expert_top10_gb300", "csrc")
    subprocess.run([cxx, "-std=c++17", "-O1", "-fPIC", "-shared", "-I", csrc, "-o", str(at / "p.so"), str(at / "p.cc")], check=True)
    f = ctypes.CDLL(str(at / "p.so")).plan

    def call(kernel, T, columns, rows, terms, sms):
        p = Plan()
        f(ctypes.byref(Kernel(*kernel)), T, columns, rows, terms, sms, ctypes.byref(p))
        return p

    return call


def walk(p, kernel, T, columns, rows, terms):
    """Every panel of one block, as the kernel lays it out and reads it."""
    tiles, warps, depth, slot, per, slabs = kernel
    chunks, split = -(-columns // per), 1 << p.log_split
    what = (kernel, T, columns, rows, terms, p.panel, split)
    assert 1 <= p.tokens <= T and p.tokens * terms <= 8 * tiles and p.grid_x >= 1 and p.grid_y >= 1, what
    assert split <= warps and p.panel >= 1 and p.panel % split == 0, what
    front = warps * (depth * slot + p.part_cols * (16 * slabs + 4) * 4) + p.tokens * p.scale_stride * 4
    assert front % 16 == 0 and p.row_stride % 16 == 0, what
    assert front + p.tokens * terms * p.row_stride <= p.bytes <= SMEM_MAX, what
    if p.pair:
        assert p.panel >= chunks and p.grid_x % 2 == 0, what
    everything = -(-columns // 32) * 32
    for first in range(0, chunks, p.panel):
        c0 = first * per
        c1 = min(c0 + p.panel * per, everything)
        # half warps lay out whole chunks; the scale of each has a place
        staged = -(-(c1 - c0) // CHUNK)
        assert c0 % CHUNK == 0, what
        assert staged <= p.scale_stride, what
        assert 2 * min(staged * CHUNK, everything - c0) <= p.row_stride, what
        # and the warps read no column that is not there: chunks of the panel, a last one in blocks of 32
        assert 2 * (c1 - c0) <= p.row_stride and c1 - c0 >= min(p.panel, chunks - first) * per - (per - 32), what


TOKENS = (1, 2, 3, 4, 5, 7, 8, 9, 10, 12, 13, 16, 17, 20, 23, 24, 25, 31, 32, 48, 49, 64, 65, 128, 145, 241, 512, 1200, 2048, 8192)
ROWS = (1, 40, 512, 1024, 2432, 2560, 4096, 10240, 12800, 32000, 32768, 131072, 1048576)


@pytest.mark.parametrize("sms", [152, 148, 20])
def test_bf16_weights(plan, sms):
    panels = 0
    for terms in (1, 2, 3):
        for T in TOKENS:
            kernel = BF16[T * terms > 8]
            for columns in (8, 40, 64, 200, 1000, 1408, 1984, 1992, 2560, 4096, 5000, 8192, 16384, 32704, 32768):
                for rows in ROWS:
                    p = plan(kernel, T, columns, rows, terms, sms)
                    walk(p, kernel, T, columns, rows, terms)
                    panels += p.panel * 64 < columns
    assert panels > 1000  # the cases that this is about are among them


@pytest.mark.parametrize("meta", [32, 64, 96, 128, 192])  # of groups of 128, 64 and 32 columns, without and with zero points
def test_4_bit_weights(plan, meta):
    one, two, more = q4_kernels(meta)
    for terms in (1, 2):
        for T in TOKENS:
            for columns in (32, 64, 96, 160, 1184, 2560, 4096, 8192, 16384, 32672, 32768):
                for rows in ROWS:
                    for kernel in (one, two) if T * terms <= 8 else (more,):
                        walk(plan(kernel, T, columns, rows, terms, 152), kernel, T, columns, rows, terms)
