"""Residual addition and RMS norm on the GPU against the fp64 oracle.

Tolerances count roundings (U = 2^-8: bf16's half step, V = 2^-24: fp32's, both
relative). The sum of H squares runs through per-thread chains, a 64-lane tree
and a chain over waves: at most CHAIN additions deep, so its relative error is
at most CHAIN V (all terms are positive); the same depth bounds signed sums
relative to the sum of their magnitudes."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_table_amd as mok
from gpu_support import DEV, host_f64
from oracle import block as B
from oracle import mxfp8
from test_gpu_dropout import TYPES, U, V, randn, rng_state

pytestmark = pytest.mark.gpu
CHAIN = 16 + 6 + 16     # 2 chunks of 8 elements a thread, 6 tree levels, 16 waves
EPS = 1e-6
SHAPES = [(1, 8), (3, 32), (5, 64), (1, 7168), (2, 1000), (33, 4096), (130, 7168), (700, 2080), (601, 128), (4, 16384),
          (520, 8200)]


def make(T, H, stream, residual, p, seed):
    x = randn((T, H), seed)
    res = randn((T, H), seed + 1, TYPES[stream], 3.0) if residual else None
    w = (1.0 + 0.25 * randn((H,), seed + 2).float()).to(torch.bfloat16)
    rng = rng_state(seed + 5, 3 * seed) if p > 0 else None
    keep = B.keep_mask(seed + 5, 3 * seed, T * H, p).reshape(T, H)
    branch = B.dropout(host_f64(x), keep, p)
    base = host_f64(res) if residual else np.zeros((T, H))
    return x, res, w, rng, keep, branch, base


def half_step(dtype):
    return U if dtype == torch.bfloat16 else V


def within(got, ref, tol, what):
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[0].tolist())


def check_mx(elems, scales, y, err):
    """Codes of a value y known to within err: the scale is that of an amax inside
    its interval, and each element rounds from a value inside its own."""
    T, H = y.shape
    sc = scales.cpu().numpy().astype(np.int64) - 127
    got = mxfp8.e4m3fn_decode(elems.cpu().numpy()).reshape(T, H // 32, 32)
    lo, hi = (np.abs(y) - err).clip(0), np.abs(y) + err
    e_lo = mxfp8.scale_exponent(lo.reshape(T, -1, 32).max(-1))
    e_hi = mxfp8.scale_exponent(hi.reshape(T, -1, 32).max(-1))
    assert ((sc >= e_lo) & (sc <= e_hi)).all()
    f = np.ldexp(1.0, -sc)[..., None]
    enc = lambda v: mxfp8.e4m3fn_decode(mxfp8.e4m3fn_encode(v.reshape(T, -1, 32) * f))  # noqa: E731
    assert ((got >= enc(y - err)) & (got <= enc(y + err))).all()


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("stream,residual,p", [("bf16", True, 0.0), ("fp32", True, 0.2), ("bf16", False, 0.3),
                                               ("fp32", False, 0.0)])
def test_forward_matches_the_oracle(T, H, stream, residual, p):
    print(f"[norm] forward T={T} H={H} {stream} residual={residual} p={p}", flush=True)
    x, res, w, rng, keep, branch, base = make(T, H, stream, residual, p, T + H)
    mx = H % 32 == 0
    r = mok.add_rmsnorm(x, w, EPS, residual=res, p=p, rng=rng, stream_dtype=TYPES[stream], mxfp8=mx)
    assert r["sum"].dtype == TYPES[stream]
    s = base + branch
    mag = np.abs(base) + np.abs(branch)
    s_err = 2 * V * mag                     # scale and one fused multiply-add
    within(host_f64(r["sum"]), s, s_err + half_step(TYPES[stream]) * np.abs(s), "sum")
    y, rstd = B.rmsnorm(s, host_f64(w), EPS)
    # mean of squares: CHAIN roundings and each square's own error; then 1/H, + eps, sqrt and the division
    ms_err = (CHAIN + 4) * V + 2 * np.sum(np.abs(s) * s_err, axis=1) / np.maximum(np.sum(s * s, axis=1), 1e-300)
    r_err = 0.5 * ms_err + 4 * V
    within(host_f64(r["rstd"]), rstd, 1.01 * r_err * rstd, "rstd")
    y_err = 1.01 * ((r_err[:, None] + 3 * V) * np.abs(y) + s_err * rstd[:, None] * np.abs(host_f64(w)))
    within(host_f64(r["y"]), y, y_err + U * np.abs(y) * 1.01, "y")
    if mx:
        check_mx(r["y_elems"], r["y_scales"], y, y_err)
        only = mok.add_rmsnorm(x, w, EPS, residual=res, p=p, rng=rng, stream_dtype=TYPES[stream], y=False, mxfp8=True)
        assert "y" not in only
        for n in ("sum", "rstd", "y_elems", "y_scales"):
            assert torch.equal(only[n], r[n]), n


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("stream,dsum,p", [("bf16", True, 0.0), ("fp32", True, 0.2), ("bf16", False, 0.3),
                                           ("fp32", False, 0.0)])
def test_backward_matches_the_oracle(T, H, stream, dsum, p):
    print(f"[norm] backward T={T} H={H} {stream} dsum={dsum} p={p}", flush=True)
    seed = 3 * T + H
    s = randn((T, H), seed, TYPES[stream], 2.0)
    w = (1.0 + 0.25 * randn((H,), seed + 1).float()).to(torch.bfloat16)
    dy = randn((T, H), seed + 2)
    ds_in = randn((T, H), seed + 3, TYPES[stream]) if dsum else None
    rstd = torch.rsqrt(s.double().square().mean(1) + EPS).float()
    rng = rng_state(seed + 4, seed) if p > 0 else None
    g = mok.add_rmsnorm_backward(dy, s, w, rstd, dsum=ds_in, p=p, rng=rng)
    S, W, D, R = (host_f64(t) for t in (s, w, dy, rstd))
    E = host_f64(ds_in) if dsum else None
    ds, dw = B.rmsnorm_backward(D, S, W, R, E)
    # |c| relative to the sum of magnitudes, then a handful of products and sums
    r = R[:, None]
    c_mag = np.mean(np.abs(D * W * S), axis=1, keepdims=True) * r * r
    mag = r * (np.abs(D * W) + np.abs(S) * c_mag) + (np.abs(E) if dsum else 0)
    err = (CHAIN + 10) * V * mag
    within(host_f64(g["dresidual"]), ds, err + half_step(TYPES[stream]) * (np.abs(ds) + err), "dresidual")
    keep = B.keep_mask(seed + 4, seed, T * H, p).reshape(T, H)
    k = 1.0 / (1.0 - p)
    within(host_f64(g["dx"]), B.dropout(ds, keep, p), k * err + U * k * (np.abs(ds) + err) * 1.01, "dx")
    # dweight: rows in chains of at most T per workgroup, then the workgroups' shares
    terms = np.sum(np.abs(D * S * r), axis=0)
    within(host_f64(g["dweight"]), dw, (T + 90) * V * terms, "dweight")
    assert g["dweight"].dtype == torch.float32
    if p == 0 and stream == "bf16":
        assert g["dx"] is g["dresidual"]


def test_gradients_are_directional_derivatives():
    T, H, p = 7, 256, 0.25
    x, res, w, rng, keep, branch, base = make(T, H, "fp32", True, p, 91)
    r = mok.add_rmsnorm(x, w, EPS, residual=res, p=p, rng=rng)
    dy, de = randn((T, H), 92), randn((T, H), 93, torch.float32)
    g = mok.add_rmsnorm_backward(dy, r["sum"], w, r["rstd"], dsum=de, p=p, rng=rng)
    D, E, W = host_f64(dy), host_f64(de), host_f64(w)
    gen = np.random.default_rng(5)

    def loss(xx, rr, ww):
        s = rr + B.dropout(xx, keep, p)
        return float(np.sum(B.rmsnorm(s, ww, EPS)[0] * D) + np.sum(s * E))

    X, Rr, h = host_f64(x), host_f64(res), 1e-5
    for name, i in (("dx", 0), ("dresidual", 1), ("dweight", 2)):
        got = host_f64(g[name])
        v = gen.standard_normal(got.shape)
        args = [X, Rr, W]
        up, dn = list(args), list(args)
        up[i], dn[i] = args[i] + h * v, args[i] - h * v
        diff = (loss(*up) - loss(*dn)) / (2 * h)
        # per element at most U relative (bf16 dx) or ~60 V of the terms; central differences are off by O(h^2)
        tol = (U if name == "dx" else 2.0 ** -16) * np.sum(np.abs(got * v)) + 1e-5 * (1 + abs(diff))
        assert abs(diff - np.sum(got * v)) <= tol, name


def test_zero_rows_and_special_values_stay_in_their_rows():
    T, H = 6, 256
    x, w = randn((T, H), 41), torch.ones(H, dtype=torch.bfloat16, device=DEV)
    ref = mok.add_rmsnorm(x, w, EPS, mxfp8=True)
    bad = x.clone()
    bad[1], bad[3, 7], bad[4, 200] = 0, float("nan"), float("inf")
    got = mok.add_rmsnorm(bad, w, EPS, mxfp8=True)
    for n in ("sum", "y", "y_elems", "y_scales", "rstd"):
        for t in (0, 2, 5):
            assert torch.equal(got[n][t], ref[n][t]), (n, t)
    assert (got["y"][1] == 0).all() and (got["y_elems"][1] & 0x7F == 0).all() and (got["y_scales"][1] == 127).all()
    assert torch.isnan(got["y"][3]).all()
    dy = randn((T, H), 42)
    g = mok.add_rmsnorm_backward(dy, bad, w, got["rstd"])
    h = mok.add_rmsnorm_backward(dy, x, w, ref["rstd"])
    for t in (0, 2, 5):
        assert torch.equal(g["dresidual"][t], h["dresidual"][t])
    assert torch.isfinite(g["dresidual"][1]).all()


def test_masked_special_values_vanish():
    T, H, p = 5, 512, 0.5
    x, res, w, rng, keep, _, _ = make(T, H, "bf16", True, p, 51)
    clean = mok.add_rmsnorm(x, w, EPS, residual=res, p=p, rng=rng)
    x[~torch.from_numpy(keep).to(DEV)] = float("nan")
    got = mok.add_rmsnorm(x, w, EPS, residual=res, p=p, rng=rng)
    for n in clean:
        assert torch.equal(got[n], clean[n]), n


def test_sum_has_the_bits_of_dropout_with_residual():
    T, H, p = 37, 1024, 0.3
    for stream in TYPES:
        x, res, w, rng, _, _, _ = make(T, H, stream, True, p, 61)
        r = mok.add_rmsnorm(x, w, EPS, residual=res, p=p, rng=rng)
        assert torch.equal(r["sum"], mok.dropout(x, rng, p, residual=res))


def test_in_place_and_neighbours_untouched():
    T, H, p = 9, 320, 0.2
    x, res, w, rng, _, _, _ = make(T, H, "bf16", True, p, 71)
    ref = mok.add_rmsnorm(x, w, EPS, residual=res, p=p, rng=rng)
    buf = torch.full(((T + 3) * H,), 7.0, dtype=torch.bfloat16, device=DEV)
    rs = buf[:T * H].view(T, H)
    rs.copy_(res)
    ybuf = torch.full((T + 3, H), 7.0, dtype=torch.bfloat16, device=DEV)
    rstd = torch.full((T + 5,), 7.0, device=DEV)
    outs = dict(sum=rs, y=ybuf[:T], rstd=rstd[:T])
    mok.add_rmsnorm(x, w, EPS, residual=rs, p=p, rng=rng, outs=outs)
    assert torch.equal(rs, ref["sum"]) and torch.equal(ybuf[:T], ref["y"]) and torch.equal(rstd[:T], ref["rstd"])
    assert (buf[T * H:] == 7.0).all() and (ybuf[T:] == 7.0).all() and (rstd[T:] == 7.0).all()
    dy, de = randn((T, H), 72), randn((T, H), 73)
    want = mok.add_rmsnorm_backward(dy, ref["sum"], w, ref["rstd"], dsum=de, p=p, rng=rng)
    want = {n: t.clone() for n, t in want.items()}
    a, b = de.clone(), dy.clone()
    got = mok.add_rmsnorm_backward(b, ref["sum"], w, ref["rstd"], dsum=a, p=p, rng=rng,
                                   grads=dict(dresidual=a, dx=b, dweight=torch.empty(H, device=DEV)))
    for n in want:
        assert torch.equal(got[n], want[n]), n


def test_no_rows():
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    e = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    r = mok.add_rmsnorm(e, w, EPS, mxfp8=True)
    assert r["y"].shape == (0, 64)
    g = mok.add_rmsnorm_backward(e, e, w, r["rstd"])
    torch.cuda.synchronize()
    assert (g["dweight"] == 0).all()


def test_repeats_streams_and_graphs_give_the_same_bits():
    T, H, p = 1100, 1536, 0.1          # more rows than workgroups in the backward
    x, res, w, rng, _, _, _ = make(T, H, "bf16", True, p, 81)
    dy, de = randn((T, H), 82), randn((T, H), 83)
    need = torch.empty(1100 * 1536 * 4, dtype=torch.uint8, device=DEV)
    need.fill_(255)                     # a workspace full of NaNs

    def step(outs=None, grads=None):
        r = mok.add_rmsnorm(x, w, EPS, residual=res, p=p, rng=rng, mxfp8=True, outs=outs)
        return r, mok.add_rmsnorm_backward(dy, r["sum"], w, r["rstd"], dsum=de, p=p, rng=rng, grads=grads,
                                           workspace=need)

    r0, g0 = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        r1, g1 = step()
    s.synchronize()
    outs, grads = {n: torch.zeros_like(t) for n, t in r0.items()}, {n: torch.zeros_like(t) for n, t in g0.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(outs, grads)
    for rep in range(3):
        for t in (*outs.values(), *grads.values()):
            t.zero_()
        step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in r0:
            assert torch.equal(outs[n], r0[n]) and torch.equal(r1[n], r0[n]), (rep, n)
        for n in g0:
            assert torch.equal(grads[n], g0[n]) and torch.equal(g1[n], g0[n]), (rep, n)
