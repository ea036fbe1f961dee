"""Quantization into blocks of 128 and the gated activation's gradient on the GPU, against fp64."""
import pytest
import torch

import mixture_experts_layer_table_amd as mok
import routed_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def _check(el, sc, v, tile, slack):
    """Codes and scales of v [B, rows, K] fp64; slack: relative error of the values that were quantized, per value."""
    s, u = R.scales(v, tile)
    assert sc.shape == s.shape and el.shape == v.shape
    worst = slack.max() if isinstance(slack, torch.Tensor) else slack
    assert ((sc.double() - s).abs() <= s * (2.0 ** -24 + worst) * 1.01).all()
    # the factor 448 / m and the product are rounded once each (2^-24), and m itself carries the slack
    off = (R.codes(el) - u).abs() - R.half_step(u) - u.abs() * (2.0 ** -23 + slack + worst) * 1.01
    assert (off <= 0).all(), float(off.max())


def _source(B, n, K, dtype, seed=0):
    g = torch.Generator().manual_seed(n * 13 + K + seed)
    v = torch.randn(B, n, K, generator=g)
    v *= torch.exp(4 * torch.randn(B, n, 1, generator=g))     # rows of different sizes
    v[:, n // 2] = 0.0
    return v.to(dtype).to(DEV)


SHAPES = [(1, 1, 16), (1, 1, 7168), (1, 5, 128), (2, 17, 144), (1, 128, 256), (3, 130, 400), (1, 1000, 1040),
          (2, 64, 2048)]


@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_rows_and_tiles(shape, dtype, tile):
    print(f"[quantize] {shape} {dtype} {tile}", flush=True)
    v = _source(*shape, dtype)
    el, sc = mok.fp8_quantize(v, tile=tile)
    _check(el, sc, v.double(), tile, 0.0)
    # the transpose of the transpose: the same bits
    if shape[1] % 8 == 0:
        el2, sc2 = mok.fp8_quantize(v.transpose(1, 2).contiguous(), True, tile=tile)
        assert torch.equal(el, el2) and torch.equal(sc, sc2)


@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,rows,K", [(1, 8, 16), (2, 72, 144), (1, 136, 272), (1, 1040, 2000), (3, 128, 128)])
def test_turned(B, rows, K, dtype, tile):
    v = _source(B, K, rows, dtype, 5)
    el, sc = mok.fp8_quantize(v, True, tile=tile)
    _check(el, sc, v.double().transpose(1, 2), tile, 0.0)


@pytest.mark.parametrize("turned", [False, True])
@pytest.mark.parametrize("rows,K", [(1, 64), (16, 16), (40, 2048), (2047, 272), (136, 144)])
def test_gated(rows, K, turned):
    if turned and rows % 8:
        pytest.skip("a turned source has rows of a multiple of 8")
    g = torch.Generator().manual_seed(rows + K)
    h = (torch.randn((1, K, 2 * rows) if turned else (1, rows, 2 * K), generator=g) * 3).to(BF).to(DEV)
    el, sc = mok.fp8_quantize(h, turned, glu=True)
    a, gate = R.glu(h), h.double().chunk(2, -1)[0]
    if turned:
        a, gate = a.transpose(1, 2), gate.transpose(1, 2)
    # e^-g through exp2: the exponent's rounding makes |g| 2^-24, exp2, the sum, the reciprocal and two products 2^-24
    # or 2^-23 each
    _check(el, sc, a, False, (gate.abs() + 12) * 2.0 ** -23)


@pytest.mark.parametrize("turned", [False, True])
@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), float("-inf")])
def test_a_block_with_no_number_is_nan_throughout(what, tile, turned):
    v = _source(1, 256, 384, F32)
    v[0, 130, 200] = what
    src = v.transpose(1, 2).contiguous() if turned else v
    el, sc = mok.fp8_quantize(src, turned, tile=tile)
    clean, csc = mok.fp8_quantize(_source(1, 256, 384, F32).transpose(1, 2).contiguous() if turned
                                  else _source(1, 256, 384, F32), turned, tile=tile)
    hit = torch.zeros_like(el, dtype=torch.bool)
    hit[0, 128 if tile else 130:256 if tile else 131, 128:256] = True
    assert ((el[hit] & 0x7F) == 0x7F).all() and torch.equal(el[~hit], clean[~hit])
    at = (0, 1, 1) if tile else (0, 1, 130)
    assert sc[at] == 1.0
    sc[at] = csc[at]
    assert torch.equal(sc, csc)


def test_small_and_large_magnitudes():
    # below 2^-52 the scale stays put; elements keep E4M3's relative accuracy down to 2^-67
    v = torch.zeros(1, 6, 128, device=DEV)
    v[0, 0, 0], v[0, 1, :] = 2.0 ** -52, 2.0 ** -60
    v[0, 2, 5], v[0, 3, 7] = 2.0 ** -140, 3.0e38
    v[0, 4, :2] = torch.tensor([448.0, -448.0])
    el, sc = mok.fp8_quantize(v)
    _check(el, sc, v.double(), False, 0.0)
    assert sc[0, 0, 5] == torch.tensor(2.0 ** -52) / 448 and (el[0, 5] == 0).all()
    assert torch.isfinite(sc).all()


@pytest.mark.parametrize("T,I", [(1, 8), (1, 2048), (37, 136), (1001, 2048), (4099, 64)])
def test_glu_backward(T, I):
    g = torch.Generator().manual_seed(T + I)
    h, da = (torch.randn(T, 2 * I, generator=g) * 3).to(BF).to(DEV), torch.randn(T, I, generator=g).to(BF).to(DEV)
    got = mok.glu_backward(da, h)
    ref = R.glu_backward(da, h)
    hg, hu = h.double().chunk(2, 1)
    s = torch.sigmoid(hg)
    mag = torch.cat([(da.double() * hu).abs() * s * (1 + hg.abs() * (1 - s)), da.double().abs() * hg.abs() * s], 1)
    rel = ((hg.abs() + 12) * 2.0 ** -22).repeat(1, 2)    # as in test_gated, s and 1 - s both
    assert ((got.double() - ref).abs() <= R.half_eps(BF) * ref.abs() * 1.01 + rel * mag + 1e-37).all()
    same = mok.glu_backward(da, h, dh=h)
    assert same is h and torch.equal(same.view(torch.int16), got.view(torch.int16))


def test_glu_of_large_gates():
    h = torch.tensor([[100.0, -100.0, 0.0, -30.0, 30.0, 1e30, -1e30, 1.0] + [2.0] * 8], device=DEV).to(BF)
    da = torch.ones(1, 8, device=DEV).to(BF)
    got = mok.glu_backward(da, h)
    assert torch.isfinite(got).all()
    ref = R.glu_backward(da, h)
    assert ((got.double() - ref).abs() <= R.half_eps(BF) * ref.abs() * 1.01 + 1e-6).all()


def test_nothing_to_quantize():
    for shape in ((0, 4, 16), (2, 0, 16), (1, 4, 0)):
        el, sc = mok.fp8_quantize(torch.empty(shape, dtype=BF, device=DEV))
        assert el.numel() == 0
    assert mok.glu_backward(torch.empty((0, 8), dtype=BF, device=DEV),
                            torch.empty((0, 16), dtype=BF, device=DEV)).shape == (0, 16)


NAN_FORMS = [(f, d) for f in ("rows", "tile", "turned", "turned tile", "gated", "gated turned", "permuted") for d in (BF, F32)
             if d is BF or not f.startswith("gated")]


@pytest.mark.parametrize("what", [float("nan"), float("-inf")])
@pytest.mark.parametrize("form,dtype", NAN_FORMS)
def test_codes_of_a_block_with_no_number_are_7f(form, dtype, what):
    # values of both signs in a block that holds a NaN or an infinity
    v = _source(1, 128, 256, F32)
    if form.startswith("gated"):
        v = torch.cat([v.abs() + 1.0, v], 2)      # g > 0: silu(g) * u has u's sign
        v[0, 17, 256 + 40] = what
    else:
        v[0, 17, 40] = what
    v = v.to(dtype)
    if form == "permuted":
        ids = torch.zeros(128, 1, dtype=torch.int32, device=DEV)
        el = mok.permute(v[0].contiguous(), mok.sort_tokens(ids, 1), rows=False, fp8=True)["elems"][None]
    else:
        turned = "turned" in form
        src = v.transpose(1, 2).contiguous() if turned and "gated" not in form else v
        if form == "gated turned":                # [K, 2 rows]: g of all rows, then u
            src = torch.cat([v[:, :, :256].transpose(1, 2), v[:, :, 256:].transpose(1, 2)], 2).contiguous()
        el, _ = mok.fp8_quantize(src, turned, tile="tile" in form, glu="gated" in form)
    hit = torch.zeros(el.shape, dtype=torch.bool, device=DEV)
    hit[0, slice(0, 128) if "tile" in form else 17, :128] = True
    assert (el[hit] == 0x7F).all(), el[hit].unique().tolist()
    assert ((el[~hit] & 0x7F) != 0x7F).all()
