"""The feed-forward block at shapes whose plan takes every tile kernel: each
product on 128- and on 256-row tiles, whole and cut along its contraction axis,
and each combination of the gradients' launch. test_block_plan.py asserts that
these shapes, with those of test_gpu_ffn.py, reach all of them. Rows, columns
and contraction axes end inside a tile, and the reference is fp64 on the device.

Tolerances are those of test_gpu_ffn.py, where they are derived."""
import pytest
import torch

import block_reference as R
from test_gpu_dropout import U, V
from test_gpu_ffn import TOL_MX, Case

pytestmark = pytest.mark.gpu

# Narrow and wide, short and long, none a multiple of a 256-row or -column tile; then the sizes of the
# benchmark's configurations, the largest too.
SHAPES_BF16 = [(3, 2112, 640), (10983, 64, 1344), (10979, 2432, 64), (3, 21824, 192), (3, 13120, 320),
               (259, 22208, 192), (141, 11456, 1408), (4999, 1344, 1216), (1001, 4096, 1024), (2048, 7168, 2048),
               (16384, 7168, 2048)]
SHAPES_MX = [(3, 1152, 1152), (10893, 640, 640), (133, 13696, 7040), (3, 640, 7296), (3, 13184, 384), (261, 22656, 384),
             (10957, 128, 2432), (4999, 1408, 1152), (1001, 4096, 1024), (2048, 7168, 2048), (16384, 7168, 2048)]


def within(got, ref, tol, what):
    off = (got.double() - ref).abs() - tol
    bad = ~(off <= 0)
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[0].tolist())
    assert float((got.double() - ref).norm()) < 1e-2 * float(ref.norm()), what


def rel_rows(got, ref):
    """The worst row's error over the row's size."""
    return float(((got.double() - ref).norm(dim=1) / ref.norm(dim=1).clamp(min=1e-300)).max())


def rel(got, ref):
    return float((got.double() - ref).norm() / ref.norm())


def operands(c):
    return dict(x=c.x.double(), wg=c.wg.double(), wu=c.wu.double(), wd=c.wd.double())


@pytest.mark.parametrize("T,H,I", SHAPES_BF16)
@pytest.mark.parametrize("addend", [True, False])
def test_bf16_forward(T, H, I, addend):
    print(f"[ffn tiles] bf16 forward T={T} H={H} I={I} addend={addend}", flush=True)
    c = Case(T, H, I, False, T + H, addend)
    o, add = operands(c), c.add.double() if addend else None
    out, h = c.forward()
    ref, rh, ra = R.forward(**o, addend=add)
    h_err = (H + 40) * V * (o["x"].abs() @ torch.cat([o["wg"].abs(), o["wu"].abs()], 1))
    within(h, rh, h_err + U * rh.abs() * 1.01, "h")
    a_err = 1.1 * h_err[:, :I] * rh[:, I:].abs() + rh[:, :I].abs() * h_err[:, I:] + 2.0 ** -18 * ra.abs()
    tol = (ra.abs() * (U + (I + 40) * V) + a_err) @ o["wd"].abs()
    within(out, ref, 1.01 * tol + U * ref.abs() * 1.01 + (2 * V * add.abs() if addend else 0), "out")


@pytest.mark.parametrize("T,H,I", SHAPES_BF16)
@pytest.mark.parametrize("addend", [True, False])
def test_bf16_backward(T, H, I, addend):
    print(f"[ffn tiles] bf16 backward T={T} H={H} I={I} addend={addend}", flush=True)
    c = Case(T, H, I, False, T + H + 1, addend)
    o, add = operands(c), c.add.double() if addend else None
    _, h = c.forward()
    g = c.backward(h)
    hs, dy = h.double(), c.dy.double()
    r = R.backward(**o, h=hs, dy=dy, addend=add)
    da_err = (H + 40) * V * (dy.abs() @ o["wd"].abs().T) + 2.0 ** -18 * (dy @ o["wd"].T).abs()
    bound = torch.cat([1.1 * hs[:, I:].abs(), hs[:, :I].abs()], 1)
    dh_op = bound * da_err.repeat(1, 2) + U * r["dh"].abs() * 1.01
    del bound, da_err
    tol = (dh_op + (2 * I + 40) * V * r["dh"].abs()) @ torch.cat([o["wg"].abs(), o["wu"].abs()], 1).T
    tol = 1.01 * tol + U * r["dx"].abs() * 1.01 + (2 * V * add.abs() if addend else 0)
    within(g["dx"], r["dx"], tol, "dx")
    tol = 1.01 * (o["x"].abs().T @ (dh_op + (T + 40) * V * r["dh"].abs()))
    for n, part in (("dw_gate", tol[:, :I]), ("dw_up", tol[:, I:])):
        within(g[n], r[n], part + U * r[n].abs() * 1.01, n)
    tol = 1.01 * ((r["a"].abs() * (U + 2.0 ** -17 + (T + 40) * V)).T @ dy.abs())
    within(g["dw_down"], r["dw_down"], tol + U * r["dw_down"].abs() * 1.01, "dw_down")


@pytest.mark.parametrize("T,H,I", SHAPES_MX)
@pytest.mark.parametrize("addend", [True, False])
def test_mxfp8(T, H, I, addend):
    print(f"[ffn tiles] mxfp8 T={T} H={H} I={I} addend={addend}", flush=True)
    c = Case(T, H, I, True, T + H + 2, addend)
    o, add = operands(c), c.add.double() if addend else None
    out, h = c.forward()
    ref, rh, _ = R.forward(**o, addend=add, fq=R.fake_quant)
    errs = dict(out=rel(out, ref), h=rel(h, rh))
    rows = dict(out=rel_rows(out, ref), h=rel_rows(h, rh))
    del ref, rh
    g = c.backward(h)
    r = R.backward(**o, h=h.double(), dy=c.dy.double(), addend=add, fq=R.fake_quant)
    errs.update({n: rel(g[n], r[n]) for n in g})
    rows["dx"] = rel_rows(g["dx"], r["dx"])
    assert all(v < TOL_MX for v in errs.values()), errs
    assert all(v < 4 * TOL_MX for v in rows.values()), rows


@pytest.mark.parametrize("H,I", [(128, 1 << 20), (1 << 20, 128)])
def test_mxfp8_widest_rows(H, I):
    # the widest rows, as test_gpu_ffn.py has them in BF16: contraction axes of 2^20 and 2^21 values, K-tiled
    print(f"[ffn tiles] mxfp8 widest H={H} I={I}", flush=True)
    c = Case(3, H, I, True, 72)
    o = operands(c)
    out, h = c.forward()
    ref, rh, _ = R.forward(**o, addend=c.add.double(), fq=R.fake_quant)
    errs = dict(out=rel(out, ref), h=rel(h, rh))
    g = c.backward(h)
    r = R.backward(**o, h=h.double(), dy=c.dy.double(), addend=c.add.double(), fq=R.fake_quant)
    errs.update({n: rel(g[n], r[n]) for n in g})
    assert all(v < TOL_MX for v in errs.values()), errs


def test_mxfp8_longest_batch():
    # T * I * 4 one row short of 2 GiB at the narrowest width: the K-tiled rows' last offsets
    T, H, I = (1 << 22) - 1, 128, 128
    print(f"[ffn tiles] mxfp8 longest T={T}", flush=True)
    c = Case(T, H, I, True, 82)
    out, h = c.forward()
    g = c.backward(h)
    w = dict(wg=c.wg.double(), wu=c.wu.double(), wd=c.wd.double())
    dw = {n: 0.0 for n in ("dw_gate", "dw_up", "dw_down")}
    for a in range(0, T, 1 << 19):
        s = slice(a, min(a + (1 << 19), T))
        x, dy, add, hs = (t[s].double() for t in (c.x, c.dy, c.add, h))
        ref, rh, _ = R.forward(x, **w, addend=add, fq=R.fake_quant)
        r = R.backward(x, **w, h=hs, dy=dy, addend=add, fq=R.fake_quant)
        for n, got, want in (("out", out[s], ref), ("h", h[s], rh), ("dx", g["dx"][s], r["dx"])):
            # the worst of four million rows: a tie taken the other way moves one of its 128 operands by at most 2^-3 of
            # itself, and one of 4 times their rms is 4 / sqrt(128) of the row: 0.044, twice that for two
            assert rel(got, want) < TOL_MX and rel_rows(got, want) < 8 * TOL_MX, (n, a)
        for n in dw:
            dw[n] = dw[n] + r[n]
    for n in dw:
        assert rel(g[n], dw[n]) < TOL_MX, n
