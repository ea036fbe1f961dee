"""Which kernels the feed-forward tests reach. The plan (ffn_plan.cpp, host code)
is compiled as it is and asked for every shape that the GPU tests run: together
they take each product on each tile, whole and cut, every form of the gradients'
launch, and the few-rows kernels past each loop's first pass and at their limits.
A refit of the plan's constants that leaves a kernel without a test fails here."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import block_reference as R
import test_gpu_ffn as G
import test_gpu_ffn_few as F
import test_gpu_ffn_tiles as L
from oracle import block as B

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_layer_table_amd",
                    "csrc")
PRODUCTS = ("gate_up", "down", "da", "dx")
PROBE = """
#include "ffn_plan.cpp"
extern "C" int probe(int64_t T, int H, int I, int precision, int32_t *o) {
    mok::FfnPlan p;
    const int s = mok::make_ffn_plan(T, H, I, precision, &p);
    if (s != MOK_OK) return s;
    for (const mok::FfnSplit &f : {p.gate_up, p.down, p.da, p.dx}) {
        *o++ = f.bm;
        *o++ = f.splits;
    }
    *o++ = p.wgrad_bm;
    *o++ = p.grads_two;
    *o++ = p.few_runs;
    *o++ = p.few_run_rows;
    return 0;
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "probe.cpp").write_text(PROBE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(d / "probe.cpp"), "-o",
                    str(d / "probe.so")], check=True)
    lib = ctypes.CDLL(str(d / "probe.so"))
    lib.probe.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_int32)]

    def ask(T, H, I, mx):
        o = (ctypes.c_int32 * 12)()
        assert lib.probe(T, H, I, int(mx), o) == 0, (T, H, I, mx)
        p = {n: (o[2 * i], o[2 * i + 1] > 1) for i, n in enumerate(PRODUCTS)}
        return dict(p, wgrad=o[8], two=bool(o[9]), few_runs=o[10], few_run_rows=o[11])
    return ask


def tile_shapes(mx):
    return (G.SHAPES_MX + L.SHAPES_MX) if mx else (G.SHAPES_BF16 + L.SHAPES_BF16)


@pytest.mark.parametrize("mx", [False, True])
def test_every_product_runs_on_every_tile(plan, mx):
    reached = set()
    for s in tile_shapes(mx):
        p = plan(*s, mx)
        for n in ("da", "dx") if p["few_runs"] else PRODUCTS:     # few rows: the forward has kernels of its own
            reached.add((n, *p[n]))
    assert reached == {(n, bm, cut) for n in PRODUCTS for bm in (128, 256) for cut in (False, True)}


@pytest.mark.parametrize("mx", [False, True])
def test_every_launch_of_the_gradients_is_reached(plan, mx):
    reached = set()
    for s in tile_shapes(mx):
        p = plan(*s, mx)
        reached.add((p["dx"], p["wgrad"], p["two"]))
    want = {((bm, cut), w, False) for bm in (128, 256) for cut in (False, True) for w in (128, 256)}
    if not mx:      # both on 128 rows, two workgroups a unit
        want |= {((128, cut), 128, True) for cut in (False, True)}
    assert reached == want


@pytest.mark.parametrize("mx", [False, True])
def test_few_rows_past_each_first_pass_and_at_the_limits(plan, mx):
    shapes = F.PASSES_MX + F.LIMITS_MX if mx else F.PASSES_BF16 + F.LIMITS_BF16
    plans = {s: plan(*s, mx) for s in shapes}
    assert all(p["few_runs"] for p in plans.values())
    for T in (1, 2):
        of = [s for s in shapes if s[0] == T]
        assert any(t * i > 2048 for t, _, i in of)                   # the values of a that 512 threads make in one go
        assert max(t * i for t, _, i in of) == 15 * 1024 and max(h for _, h, _ in of) == 16 * 2048
        if mx:
            assert any(h > 7 * 1024 for _, h, _ in of)               # 7 pieces of 16 values by 64 lanes
        else:
            assert any(i > 16 * 128 for _, _, i in of)               # 16 loads of 128 rows of W_down
            rows = [plans[s]["few_run_rows"] for s in of]
            assert any(r > 16 * 64 for r in rows) and any(r % (16 * 64) for r in rows)
    # one step past a limit, the tiles take over
    q = 128 if mx else 64
    assert not plan(1, q, 15 * 1024 + q, mx)["few_runs"] and not plan(1, 16 * 2048 + q, q, mx)["few_runs"]
    assert not plan(3, 1024, 512, mx)["few_runs"]


def test_the_device_reference_is_the_oracle():
    T, H, I = 5, 128, 64
    gen = np.random.default_rng(1)
    x, dy, add = (gen.standard_normal((T, H)) for _ in range(3))
    wg, wu = (gen.standard_normal((H, I)) / 11 for _ in range(2))
    wd = gen.standard_normal((I, H)) / 8
    ops = dict(x=x, wg=wg, wu=wu, wd=wd, addend=add)
    t = lambda v: torch.from_numpy(v)  # noqa: E731
    for fq, rq in ((None, R.keep), (B.fake_quant, R.fake_quant)):
        want, got = B.ffn(**ops, fq=fq), R.forward(**{n: t(v) for n, v in ops.items()}, fq=rq)
        for a, b in zip(got, want):
            assert np.allclose(a.numpy(), b, rtol=1e-12, atol=1e-12)
        h = want[1]
        wb = B.ffn_backward(x, wg, wu, wd, h, dy, add, fq)
        gb = R.backward(t(x), t(wg), t(wu), t(wd), t(h), t(dy), t(add), rq)
        for n in wb:
            assert np.allclose(gb[n].numpy(), wb[n], rtol=1e-12, atol=1e-12), n


def test_the_reference_quantizer_at_the_ends_of_its_range():
    v = np.zeros((6, 32))
    v[0, :4] = [1.0, 2.0 ** -9, 3 * 2.0 ** -11, -2.0 ** -10]     # subnormal codes and a tie between two
    v[1, :3] = [480.0, 449.0, -500.0]                            # past 448 at their scale
    v[2] = np.arange(32) * 0.0625 + 1.0                          # ties in the upper binades
    v[3, 0] = 2.0 ** -130                                        # below the smallest scale
    v[4, :2] = [2.0 ** 120, -2.0 ** 100]
    bf = torch.from_numpy(v)
    assert np.array_equal(R.fake_quant(bf, 1).numpy(), B.fake_quant(v, 1))
    assert np.array_equal(R.fake_quant(bf.T.contiguous(), 0).numpy(), B.fake_quant(v.T, 0))
