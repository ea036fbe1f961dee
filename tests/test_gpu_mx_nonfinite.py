"""A NaN or an infinity on its way through MXFP8 rows: the block that holds it is
NaN throughout, the outputs of its row show a NaN, and every other row keeps its
bits. (E4M3FN's NaN is 0x7F or 0xFF; it has no infinity.)"""
import numpy as np
import pytest
import torch

import mixture_experts_layer_table_amd as mok
import synth
from gpu_support import DEV, DeviceInputs, knobs, run_layer, status_word
from test_gpu_dropout import randn
from test_gpu_ffn import Case
from test_gpu_mxfp8_layer import SMALL

pytestmark = pytest.mark.gpu
BAD = {"nan": float("nan"), "inf": float("inf"), "-inf": -float("inf")}


def is_nan(codes):
    return (codes & 0x7F) == 0x7F


def others(T, *rows):
    ok = torch.ones(T, dtype=torch.bool, device=DEV)
    ok[list(rows)] = False
    return ok


@pytest.mark.parametrize("transposed", [False, True])
def test_quantize(transposed):
    rows, K = 5, 256
    x = randn((1, rows, K), 1)
    src = (lambda t: t.transpose(1, 2).contiguous()) if transposed else (lambda t: t)
    e0, s0 = mok.mxfp8_quantize(src(x), transposed)
    bad = x.clone()
    bad[0, 1, 40], bad[0, 2, 70], bad[0, 4, 255] = BAD["nan"], BAD["inf"], BAD["-inf"]
    e, s = mok.mxfp8_quantize(src(bad), transposed)
    hit = torch.zeros((1, rows, K // 32), dtype=torch.bool, device=DEV)
    hit[0, 1, 1] = hit[0, 2, 2] = hit[0, 4, 7] = True
    wide = hit.repeat_interleave(32, 2)
    assert torch.equal(is_nan(e), wide)
    assert torch.equal(e[~wide], e0[~wide]) and torch.equal(s[~hit], s0[~hit])


@pytest.mark.parametrize("H", [64, 4096, 7168])
def test_norm_rows(H):
    T = 6
    x, w = randn((T, H), 2), torch.ones(H, dtype=torch.bfloat16, device=DEV)
    ref = mok.add_rmsnorm(x, w, 1e-6, mxfp8=True)
    bad = x.clone()
    bad[1, 7], bad[3, H - 1], bad[4, 33] = BAD["nan"], BAD["inf"], BAD["-inf"]
    got = mok.add_rmsnorm(bad, w, 1e-6, mxfp8=True)
    nan = is_nan(got["y_elems"])
    assert nan[1].all()                                  # the row's 1 / rms is NaN
    for t, c in ((3, H - 1), (4, 33)):                   # 1 / rms is 0: 0 elsewhere, NaN where infinity meets it
        at = torch.zeros(H, dtype=torch.bool, device=DEV)
        at[c // 32 * 32:c // 32 * 32 + 32] = True
        assert torch.equal(nan[t], at) and (got["y_elems"][t][~at] & 0x7F == 0).all()
        assert torch.isnan(got["y"][t, c])
    ok = others(T, 1, 3, 4)
    for n in ("sum", "y", "y_elems", "y_scales", "rstd"):
        assert torch.equal(got[n][ok], ref[n][ok]), n


# two rows (their own kernels), more; gate/up and dA whole, and cut along the hidden size
SHAPES = [(2, 1024, 512), (4, 256, 256), (300, 256, 256), (300, 4096, 256)]


@pytest.mark.parametrize("T,H,I", SHAPES)
def test_ffn_forward(T, H, I):
    print(f"[mx nonfinite] forward T={T} H={H} I={I}", flush=True)
    c = Case(T, H, I, True, 7)
    out, h = c.forward()
    e, s = (t.clone() for t in c.rows)
    e[T - 1, 5] = 0x7F                                   # a NaN that arrives with the rows
    got, gh = mok.ffn_forward(c.ws, (e, s), c.wf, addend=c.add)
    assert torch.isnan(got[T - 1]).all() and torch.isnan(gh[T - 1]).all()
    ok = others(T, T - 1)
    assert torch.equal(got[ok], out[ok]) and torch.equal(gh[ok], h[ok])
    e, s = (t.clone() for t in c.rows)
    s[0] = 254                                           # pre-activations past fp32: infinities arise in the block itself
    got, gh = mok.ffn_forward(c.ws, (e, s), c.wf, addend=c.add)
    assert not torch.isfinite(gh[0]).all() and torch.isnan(got[0]).all()
    assert torch.equal(got[1:], out[1:]) and torch.equal(gh[1:], h[1:])


@pytest.mark.parametrize("bad", list(BAD))
@pytest.mark.parametrize("T,H,I", SHAPES)
def test_ffn_backward(T, H, I, bad):
    print(f"[mx nonfinite] backward T={T} H={H} I={I} {bad}", flush=True)
    c = Case(T, H, I, True, 8)
    _, h = c.forward()
    dx = c.backward(h)["dx"]
    r = T // 2
    ok = others(T, r)
    dy = c.dy.clone()
    dy[r, H - 3] = BAD[bad]
    got = mok.ffn_backward(c.ws, c.x, c.wb, h, dy, addend=c.add)["dx"]
    assert torch.isnan(got[r]).all() and torch.equal(got[ok], dx[ok])
    bad_h = h.clone()
    bad_h[r, I + 2] = BAD[bad]                           # of h_u: dh_g = G h_u s (...) is not finite
    got = c.backward(bad_h)["dx"]
    assert torch.isnan(got[r]).all() and torch.equal(got[ok], dx[ok])


@pytest.mark.parametrize("wgrad", [False, True])
def test_routed_layer(wgrad):
    cfg = SMALL["mx_k2_ragged"]
    print(f"[mx nonfinite] routed layer wgrad={wgrad}", flush=True)
    prec = mok.MOK_MXFP8_WGRAD if wgrad else mok.MOK_MXFP8
    d = DeviceInputs(synth.make_inputs(cfg))
    want = run_layer(d, knobs(cfg, precision=prec))
    r = 17
    ok = others(cfg.T, r)
    d.x[r, 3] = BAD["nan"]
    got = run_layer(d, knobs(cfg, precision=prec))
    assert status_word(got["schedule"]) == 0
    assert torch.isnan(got["out"][r]).all() and torch.equal(got["out"][ok], want["out"][ok])
    hit = np.unique(d.ids[r].cpu().numpy())              # its experts' gate gradients read the row
    for e in range(cfg.E):
        assert bool(torch.isnan(got["dw_gate"][e]).any()) == (e in hit), e
