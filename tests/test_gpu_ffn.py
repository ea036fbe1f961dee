"""The gated feed-forward block on the GPU against the fp64 oracle, in BF16 and
MXFP8, from one row to several tiles.

BF16 tolerances count roundings element by element (U = 2^-8, V = 2^-24): an
fp32 accumulation of K products is off by at most (K + 40) V of the sum of
their magnitudes (K-step order, partials, the activation's few operations); an
operand rounded to bf16 (a, dh) adds U of that same sum; the output adds U of
itself. MXFP8 outputs are held by the relative Frobenius norm: rounding the
output adds at most U, and an operand so near a tie that fp32 and fp64 round it
apart moves by at most 2^-3 of itself; at most one in a thousand does (an
operand's relative error, about 1e-5, over E4M3's step 2^-3 to 2^-4), which adds
at most 2^-3 sqrt(1e-3) = 4e-3: together under 1e-2."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_table_amd as mok
from gpu_support import DEV, host_f64
from oracle import block as B
from oracle import layer as L
from test_gpu_dropout import U, V, randn

pytestmark = pytest.mark.gpu
TOL_MX = 1e-2

# rows around 1, 32, 128 and 256 (MFMA blocks and tile heights), widths below, at and past one tile, long
# contraction axes (split) and short ones; BF16 takes multiples of 64, MXFP8 of 128
# one and two rows take kernels of their own (more of them in test_gpu_ffn_few.py): run lengths and strips that do not
# divide evenly; the shapes that take each tile kernel are in test_gpu_ffn_tiles.py
SHAPES_BF16 = [(1, 64, 64), (1, 1024, 512), (3, 192, 320), (2, 320, 192), (4, 2112, 1088), (1, 7168, 2048),
               (4, 128, 4096), (2, 5120, 64), (31, 128, 64), (33, 640, 192), (128, 512, 448),
               (129, 320, 128), (257, 256, 640), (300, 1088, 576), (700, 64, 1024), (65, 4096, 128), (5, 7168, 2048)]
SHAPES_MX = [(1, 128, 128), (1, 1024, 512), (3, 256, 384), (2, 384, 128), (4, 2176, 1152), (1, 7168, 2048),
             (4, 128, 4096), (2, 5120, 128), (31, 128, 256), (33, 640, 256), (257, 256, 640),
             (300, 1152, 640), (700, 128, 1024), (65, 4096, 128), (5, 7168, 2048)]


class Case:
    def __init__(self, T, H, I, mx, seed=0, addend=True):
        self.T, self.H, self.I, self.mx = T, H, I, mx
        self.x, self.dy = randn((T, H), seed + 1), randn((T, H), seed + 2)
        self.wg, self.wu = randn((H, I), seed + 3, scale=H ** -0.5), randn((H, I), seed + 4, scale=H ** -0.5)
        self.wd = randn((I, H), seed + 5, scale=I ** -0.5)
        self.add = randn((T, H), seed + 6) if addend else None
        self.ws = mok.get_ffn_workspace(mok.MOK_MXFP8 if mx else mok.MOK_BF16, device=DEV, num_tokens=T, hidden_size=H,
                                        intermediate_size=I)
        self.ws.buffer.fill_(255)       # NaN in every type: nothing unwritten may reach an output
        if mx:
            w = mok.MXFP8Weights(self.wg[None], self.wu[None], self.wd[None])
            self.wf, self.wb = w.fwd, w.bwd
            self.keep = w
            e, s = mok.mxfp8_quantize(self.x[None], False)
            self.rows = (e[0], s[0])
        else:
            self.wf = self.wb = mok.weights_bf16(self.wg, self.wu, self.wd)
            self.rows = self.x

    def forward(self, **kw):
        return mok.ffn_forward(self.ws, self.rows, self.wf, addend=self.add, **kw)

    def backward(self, h, **kw):
        return mok.ffn_backward(self.ws, self.x, self.wb, h, self.dy, addend=self.add, **kw)

    def oracle(self):
        f = host_f64
        return dict(x=f(self.x), wg=f(self.wg), wu=f(self.wu), wd=f(self.wd),
                    addend=None if self.add is None else f(self.add))


def within(got, ref, tol, what):
    got = host_f64(got)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[0].tolist())
    assert L.rel_frobenius(got, ref) < 1e-2, what


@pytest.mark.parametrize("T,H,I", SHAPES_BF16)
@pytest.mark.parametrize("addend", [True, False])
def test_bf16_matches_the_oracle(T, H, I, addend):
    print(f"[ffn] bf16 T={T} H={H} I={I} addend={addend}", flush=True)
    c = Case(T, H, I, False, T + H + I, addend)
    o = c.oracle()
    out, h = c.forward()
    ref, rh, ra = B.ffn(**o)
    xw = np.abs(o["x"]) @ np.concatenate([np.abs(o["wg"]), np.abs(o["wu"])], 1)
    h_err = (H + 40) * V * xw
    within(h, rh, h_err + U * np.abs(rh) * 1.01, "h")
    # a = silu(g) u: |silu'| <= 1.1, |silu(g)| <= |g|; 2^-18 of a covers the fast exponential and reciprocal
    a_err = 1.1 * h_err[:, :I] * np.abs(rh[:, I:]) + np.abs(rh[:, :I]) * h_err[:, I:] + 2.0 ** -18 * np.abs(ra)
    aw = (np.abs(ra) * (U + (I + 40) * V) + a_err) @ np.abs(o["wd"])
    add = np.abs(o["addend"]) if addend else 0
    within(out, ref, aw * 1.01 + U * np.abs(ref) * 1.01 + 2 * V * add, "out")
    # backward from the h the forward saved
    g = c.backward(h)
    hs = host_f64(h)
    dy = host_f64(c.dy)
    r = B.ffn_backward(o["x"], o["wg"], o["wu"], o["wd"], hs, dy, o["addend"])
    da_err = (H + 40) * V * (np.abs(dy) @ np.abs(o["wd"]).T)
    da = np.abs(dy @ o["wd"].T)
    hg, hu = hs[:, :I], hs[:, I:]
    # dh = da * f(h): |f_g| <= 1.1 |h_u|, |f_u| <= |h_g|, evaluated to 2^-18 of da times those bounds
    dh_err = np.concatenate([1.1 * np.abs(hu), np.abs(hg)], 1) * np.tile(da_err + 2.0 ** -18 * da, 2)
    dh_op = dh_err + U * np.abs(r["dh"]) * 1.01            # as a bf16 operand
    wcat = np.abs(np.concatenate([o["wg"], o["wu"]], 1))
    tol = (dh_op + (2 * I + 40) * V * np.abs(r["dh"])) @ wcat.T + U * np.abs(r["dx"]) * 1.01 + 2 * V * add
    within(g["dx"], r["dx"], 1.01 * tol, "dx")
    tol = np.abs(o["x"]).T @ (dh_op + (T + 40) * V * np.abs(r["dh"]))
    dw = np.concatenate([r["dw_gate"], r["dw_up"]], 1)
    tol = 1.01 * tol + U * np.abs(dw) * 1.01
    within(g["dw_gate"], r["dw_gate"], tol[:, :I], "dw_gate")
    within(g["dw_up"], r["dw_up"], tol[:, I:], "dw_up")
    tol = (np.abs(r["a"]) * (U + 2.0 ** -17 + (T + 40) * V)).T @ np.abs(dy)
    within(g["dw_down"], r["dw_down"], 1.01 * tol + U * np.abs(r["dw_down"]) * 1.01, "dw_down")


@pytest.mark.parametrize("T,H,I", SHAPES_MX)
@pytest.mark.parametrize("addend", [True, False])
def test_mxfp8_matches_the_fake_quant_oracle(T, H, I, addend):
    print(f"[ffn] mxfp8 T={T} H={H} I={I} addend={addend}", flush=True)
    c = Case(T, H, I, True, T + H + I, addend)
    o = c.oracle()
    out, h = c.forward()
    ref, rh, _ = B.ffn(fq=B.fake_quant, **o)
    hs, dy = host_f64(h), host_f64(c.dy)
    g = c.backward(h)
    r = B.ffn_backward(o["x"], o["wg"], o["wu"], o["wd"], hs, dy, o["addend"], B.fake_quant)
    errs = dict(h=L.rel_frobenius(hs, rh), out=L.rel_frobenius(host_f64(out), ref))
    errs.update({n: L.rel_frobenius(host_f64(g[n]), r[n]) for n in g})
    rows = {n: float(np.max(L.rel_rows(a, b))) for n, a, b in (("out", host_f64(out), ref), ("h", hs, rh),
                                                               ("dx", host_f64(g["dx"]), r["dx"]))}
    assert all(v < TOL_MX for v in errs.values()), errs
    assert all(v < 4 * TOL_MX for v in rows.values()), rows   # a row averages fewer ties: twice the bound, doubled


def test_gradients_are_directional_derivatives():
    c = Case(37, 256, 192, False, 9)
    o = c.oracle()
    _, h = c.forward()
    g = c.backward(h)
    dy = host_f64(c.dy)
    gen = np.random.default_rng(3)
    names = dict(x="dx", wg="dw_gate", wu="dw_up", wd="dw_down")
    for k, n in names.items():
        v = gen.standard_normal(o[k].shape)
        eps = 1e-5
        lo, hi = dict(o), dict(o)
        lo[k], hi[k] = o[k] - eps * v, o[k] + eps * v
        diff = float(np.sum((B.ffn(**hi)[0] - B.ffn(**lo)[0]) * dy)) / (2 * eps)
        got = host_f64(g[n]) - (host_f64(c.add) if n == "dx" else 0)
        # roundings of h, dh or a and of the gradient itself, 3 U an element at most, random signs over the sum:
        # bounded by 3 U of the sum's Euclidean norm times 5
        tol = 3 * U * 5 * np.linalg.norm(got * v) + 1e-4 * abs(diff)
        assert abs(diff - np.sum(got * v)) <= tol, (n, diff, float(np.sum(got * v)))


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T", [1, 3, 5, 300, 513])
def test_no_h_in_place_and_neighbours_untouched(mx, T):
    H, I = 512, 384
    c = Case(T, H, I, mx, 21)
    out, h = c.forward()
    want, _ = c.forward(save_h=False)
    assert torch.equal(out, want)
    buf = torch.full((T + 2, H), 9.0, dtype=torch.bfloat16, device=DEV)
    buf[:T] = c.add
    mok.ffn_forward(c.ws, c.rows, c.wf, addend=buf[:T], out=buf[:T], save_h=False)
    assert torch.equal(buf[:T], out) and (buf[T:] == 9.0).all()
    g = c.backward(h)
    buf[:T] = c.add
    big = {n: torch.full((t.shape[0] + 2, t.shape[1]), 9.0, dtype=t.dtype, device=DEV) for n, t in g.items()}
    grads = {n: t[:-2] for n, t in big.items()}
    grads["dx"] = buf[:T]
    mok.ffn_backward(c.ws, c.x, c.wb, h, c.dy, addend=buf[:T], grads=grads)
    for n in g:
        assert torch.equal(grads[n], g[n]), n
        if n != "dx":
            assert (big[n][-2:] == 9.0).all(), n
    assert (buf[T:] == 9.0).all()


@pytest.mark.parametrize("T", [2, 4, 7, 300])
def test_special_values_stay_in_their_row(T):
    c = Case(T, 256, 192, False, 31)
    out, h = c.forward()
    a, b = (0, 1) if T == 2 else (1, 3) if T == 4 else (3, 4)
    c.x[a, 5], c.x[b, 200] = float("nan"), float("inf")
    got, gh = c.forward()
    ok = torch.ones(T, dtype=torch.bool, device=DEV)
    ok[a] = ok[b] = False
    assert torch.equal(got[ok], out[ok]) and torch.equal(gh[ok], h[ok])
    assert torch.isnan(got[a]).all()
    g0 = c.backward(h)["dx"].clone()
    h[a] = float("nan")
    assert torch.equal(c.backward(h)["dx"][ok], g0[ok])


@pytest.mark.parametrize("mx", [False, True])
def test_fewer_rows_in_a_larger_workspace(mx):
    c = Case(300, 512, 256, mx, 41)
    small = Case(40, 512, 256, mx, 41)
    rows = tuple(t[:40] for t in c.rows) if mx else c.rows[:40]
    small.wf, small.wb = c.wf, c.wb
    small.rows, small.x, small.dy, small.add = rows, c.x[:40], c.dy[:40], c.add[:40]
    out, h = small.forward()
    want, wh = mok.ffn_forward(c.ws, rows, c.wf, addend=c.add[:40])
    assert torch.equal(out, want) and torch.equal(h, wh)
    g = small.backward(h)
    w = mok.ffn_backward(c.ws, c.x[:40], c.wb, h, c.dy[:40], addend=c.add[:40])
    for n in g:
        assert torch.equal(g[n], w[n]), n


@pytest.mark.parametrize("mx", [False, True])
def test_no_rows(mx):
    c = Case(0, 256, 128, mx, 51, addend=False) if not mx else None
    if mx:
        full = Case(4, 256, 128, True, 51)
        rows = tuple(t[:0] for t in full.rows)
        out, h = mok.ffn_forward(full.ws, rows, full.wf)
        g = mok.ffn_backward(full.ws, full.x[:0], full.wb, h, full.dy[:0])
    else:
        out, h = c.forward()
        g = c.backward(h)
    torch.cuda.synchronize()
    assert out.shape == (0, 256) and all((g[n] == 0).all() for n in ("dw_gate", "dw_up", "dw_down"))


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T", [3, 520])
def test_repeats_streams_and_graphs_give_the_same_bits(mx, T):
    c = Case(T, 1024, 512, mx, 61)
    out0, h0 = c.forward()
    g0 = c.backward(h0)
    ref = dict(out=out0.clone(), h=h0.clone(), **{n: t.clone() for n, t in g0.items()})
    for _ in range(5):
        out, h = c.forward()
        for n, t in dict(out=out, h=h, **c.backward(h)).items():
            assert torch.equal(t, ref[n]), n
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out, h = c.forward()
        g = c.backward(h)
    s.synchronize()
    for n, t in dict(out=out, h=h, **g).items():
        assert torch.equal(t, ref[n]), n
    got = {n: torch.empty_like(t) for n, t in ref.items()}
    grads = {n: got[n] for n in g0}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.forward(out=got["out"], h=got["h"])
        c.backward(got["h"], grads=grads)
    for rep in range(3):
        for t in got.values():
            t.zero_()
        c.forward()          # eager work through the same workspace between replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n, t in ref.items():
            assert torch.equal(got[n], t), (rep, n)


@pytest.mark.parametrize("T", [1, 2])
def test_block_scales_far_apart(T):
    # 2^100 taken from the weights' scales and given to the rows': the same products
    c = Case(T, 1024, 512, True, 65)
    out, h = c.forward()
    e, s = c.rows
    q = c.keep
    assert int(s.max()) <= 154 and int(q.fwd_gate[1].min()) >= 101 and int(q.fwd_up[1].min()) >= 101
    w = mok.weights_mxfp8((q.fwd_gate[0], q.fwd_gate[1] - 100), (q.fwd_up[0], q.fwd_up[1] - 100), q.fwd_down, "fwd")
    out2, h2 = mok.ffn_forward(c.ws, (e, s + 100), w, addend=c.add)
    assert torch.equal(h, h2) and torch.equal(out, out2)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T", [1, 65, 520])
def test_two_streams_at_once(mx, T):
    # each with its own workspace, beside each other with no wait between them
    a, b = Case(T, 1024, 512, mx, 66), Case(T, 1024, 512, mx, 67)
    want = []
    for c in (a, b):
        out, h = c.forward()
        want.append(dict(out=out, h=h, **c.backward(h)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(10):
        for c, s, g in zip((a, b), streams, got):
            with torch.cuda.stream(s):
                out, h = c.forward()
                g.append(dict(out=out, h=h, **c.backward(h)))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for r in g:
            for n, t in w.items():
                assert torch.equal(r[n], t), n


@pytest.mark.parametrize("H,I", [(64, 1 << 20), (1 << 20, 64)])
def test_widest_shapes(H, I):
    # the widest rows: offsets of rows past the tile's valid ones reach 2^32 and must not wrap into them
    T = 3
    print(f"[ffn] widest T={T} H={H} I={I}", flush=True)
    c = Case(T, H, I, False, 71)
    o = c.oracle()
    out, h = c.forward()
    ref, rh, _ = B.ffn(**o)
    g = c.backward(h)
    r = B.ffn_backward(o["x"], o["wg"], o["wu"], o["wd"], host_f64(h), host_f64(c.dy), o["addend"])
    errs = dict(out=L.rel_frobenius(host_f64(out), ref), h=L.rel_frobenius(host_f64(h), rh))
    errs.update({n: L.rel_frobenius(host_f64(g[n]), r[n]) for n in g})
    assert all(v < 1e-2 for v in errs.values()), errs


def test_longest_batch():
    # T * I * 4 one row short of 2 GiB: the largest batch the offsets allow, at the narrowest width
    T, H, I = (1 << 23) - 1, 64, 64
    print(f"[ffn] longest T={T}", flush=True)
    c = Case(T, H, I, False, 81)
    out, h = c.forward()
    g = c.backward(h)
    pick = torch.cat([torch.arange(0, 300), torch.arange(T // 2 - 150, T // 2 + 150), torch.arange(T - 300, T)]).to(DEV)
    f = lambda t: host_f64(t[pick])  # noqa: E731
    wg, wu, wd = (host_f64(w) for w in (c.wg, c.wu, c.wd))
    ref, rh, _ = B.ffn(f(c.x), wg, wu, wd, f(c.add))
    r = B.ffn_backward(f(c.x), wg, wu, wd, f(h), f(c.dy), f(c.add))
    for got, want in ((f(out), ref), (f(h), rh), (f(g["dx"]), r["dx"])):
        assert float(np.max(L.rel_rows(got, want))) < 2e-2
    # weight gradients over all rows, in fp64 chunk by chunk on the device
    dw = {n: torch.zeros(g[n].shape, dtype=torch.float64, device=DEV) for n in ("dw_gate", "dw_up", "dw_down")}
    for a in range(0, T, 1 << 20):
        x, dy, hh = (t[a:a + (1 << 20)].double() for t in (c.x, c.dy, h))
        hg, hu = hh[:, :I], hh[:, I:]
        s = torch.sigmoid(hg)
        da = dy @ c.wd.double().T
        dw["dw_gate"] += x.T @ (da * hu * s * (1 + hg * (1 - s)))
        dw["dw_up"] += x.T @ (da * hg * s)
        dw["dw_down"] += (hg * s * hu).T @ dy
    # fp32 sums of 2^23 products: random roundings, about 2^-24 sqrt(2^23) of the sum's size, beside bf16's 2^-8
    for n, want in dw.items():
        assert float((g[n].double() - want).norm() / want.norm()) < 1e-2, n
