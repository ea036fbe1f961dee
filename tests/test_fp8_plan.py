"""The plan of the products on blocks of 128, compiled for the host: the GPU tests'
shapes take every path, and every plan is one that the kernels can run (CPU)."""
import ctypes
import os
import subprocess

import pytest

import fp8_shapes as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixture_experts_layer_table_amd", "csrc")


class Shape(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("E", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32)]


class Plan(ctypes.Structure):
    _fields_ = [("bm", ctypes.c_int32), ("few", ctypes.c_int32), ("splits", ctypes.c_int32), ("run", ctypes.c_int32),
                ("total", ctypes.c_size_t), ("few_w", ctypes.c_int32)]


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, lib = d / "plan.cpp", d / "plan.so"
    src.write_text(f'''#include "{CSRC}/fp8_plan.h"
struct Out {{ int32_t bm, few, splits, run; size_t total; int32_t few_w; }};
extern "C" int plan(int wgrad, const mok_fp8_shape *s, Out *o) {{
    mok::BlkPlan p;
    const int r = wgrad ? mok::make_blk_wgrad_plan(s, &p) : mok::make_blk_matmul_plan(s, &p);
    if (r == 0) *o = Out{{p.bm, p.few, p.splits, p.run, p.total, p.few_w}};
    return r;
}}
''')
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", str(src), os.path.join(CSRC, "fp8_plan.cpp"), "-o",
                    str(lib)], check=True)
    f = ctypes.CDLL(str(lib)).plan

    def call(wgrad, M, N, K, E, f32):
        p = Plan()
        status = f(int(wgrad), ctypes.byref(Shape(M, N, K, E, int(f32))), ctypes.byref(p))
        assert status in (0, 2)          # 2: more tiles than one grid holds
        return p if status == 0 else None
    return call


@pytest.mark.parametrize("name", list(S.DENSE))
def test_dense_shapes_take_their_path(plan, name):
    M, N, K, f32, (few, bm, runs) = S.DENSE[name]
    p = plan(False, M, N, K, 0, f32)
    assert (p.few, p.bm) == (few, bm) and (p.splits == runs if runs else p.splits > 1)


@pytest.mark.parametrize("name", list(S.GROUPED))
def test_grouped_shapes_take_their_path(plan, name):
    rows, N, K, f32, (few, bm, runs) = S.GROUPED[name]
    p = plan(False, sum(rows), N, K, len(rows), f32)
    assert (p.few, p.bm) == (few, bm) and (p.splits == runs if runs else p.splits > 1)


def test_few_rows_take_both_widths(plan):
    for shapes, grouped in ((S.DENSE, False), (S.GROUPED, True)):
        for name, (rows, N, K, f32, (few, _, _)) in shapes.items():
            p = plan(False, sum(rows) if grouped else rows, N, K, len(rows) if grouped else 0, f32)
            assert p.few_w == (0 if few == 0 else 2 if "wide" in name else 1), name


@pytest.mark.parametrize("name", list(S.WGRAD))
def test_weight_gradient_shapes_take_their_path(plan, name):
    N, K, rows, f32, (bm, runs) = S.WGRAD[name]
    M, E = (sum(rows), len(rows)) if isinstance(rows, list) else (rows, 0)
    p = plan(True, M, N, K, E, f32)
    assert p.bm == bm and (p.splits == runs if runs else p.splits > 1)


def test_every_plan_can_run(plan):
    for f32 in (False, True):
        for E in (0, 1, 3, 64, 4096):
            for M in (0, 1, 16, 48, 272, 1024, 4112, 65536, 1 << 22):
                for N, K in ((16, 16), (144, 1040), (4096, 7168), (1 << 16, 128), (128, 1 << 20)):
                    p = plan(False, M, N, K, E, f32)
                    if p is None:
                        assert (M // 128 + E) * (N // 256) >= 1 << 22
                        continue
                    kb = -(-K // 128)
                    assert p.bm in (128, 256) and p.few in (0, 1, 2, 4) and (p.total > 0) == (p.splits > 1)
                    assert not (f32 and p.bm == 256)
                    if p.splits > 1:
                        assert p.bm == 128 and p.few == 0 and -(-kb // p.run) == p.splits
                        assert p.total == p.splits * M * N * 4 <= 64 << 20
                    if p.few:
                        assert (min(E, M) if E else 1) * N // 16 * 512 < 1 << 32
                    if M % 16 == 0 and M < 1 << 22:
                        w = plan(True, M, N, K, E, f32)
                        if w is None:
                            assert max(E, 1) * (N // 128 + 1) * (K // 256 + 1) >= 1 << 22
                            continue
                        assert w.bm in (128, 256) and (w.splits == 1 or w.total == w.splits * max(E, 1) * N * K * 4)
                        assert w.total <= 64 << 20 and not (f32 and w.bm == 256)
