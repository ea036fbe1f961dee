"""Forms of the residual RMS norm that a caller may choose: gradient buffers of
its own, and outputs left out through the C ABI. Which buffers a call gets never
changes what it computes, so every form is held to the bits of the full one."""
import pytest
import torch

import mixture_experts_layer_table_amd as mok
from gpu_support import DEV
from test_gpu_dropout import TYPES, randn, rng_state

pytestmark = pytest.mark.gpu
T, H, EPS = 37, 512, 1e-6


def backward_inputs(stream):
    s, dy = randn((T, H), 1, TYPES[stream], 2.0), randn((T, H), 2)
    w = (1.0 + 0.25 * randn((H,), 3).float()).to(torch.bfloat16)
    rstd = torch.rsqrt(s.double().square().mean(1) + EPS).float()
    return dy, s, w, rstd, randn((T, H), 4, TYPES[stream])


@pytest.mark.parametrize("stream,p", [("bf16", 0.0), ("bf16", 0.25), ("fp32", 0.0)])
def test_a_given_dx_is_written(stream, p):
    # a loop with static buffers reads its dx whatever p has become
    dy, s, w, rstd, dsum = backward_inputs(stream)
    rng = rng_state(5, 6) if p > 0 else None
    want = mok.add_rmsnorm_backward(dy, s, w, rstd, dsum=dsum, p=p, rng=rng)
    grads = dict(dresidual=torch.full_like(s, 7.0), dx=torch.full_like(dy, 7.0),
                 dweight=torch.full((H,), 7.0, device=DEV))
    got = mok.add_rmsnorm_backward(dy, s, w, rstd, dsum=dsum, p=p, rng=rng, grads=grads)
    for n in ("dresidual", "dx", "dweight"):
        assert got[n] is grads[n] and torch.equal(grads[n], want[n]), n


def test_the_returned_gradients_serve_as_buffers():
    # bf16 and p == 0: the dict holds one tensor under two names, and may come back as grads
    dy, s, w, rstd, dsum = backward_inputs("bf16")
    first = mok.add_rmsnorm_backward(dy, s, w, rstd, dsum=dsum)
    want = {n: t.clone() for n, t in first.items()}
    for t in first.values():
        t.zero_()
    again = mok.add_rmsnorm_backward(dy, s, w, rstd, dsum=dsum, grads=first)
    assert again["dx"].data_ptr() == again["dresidual"].data_ptr()
    for n in want:
        assert torch.equal(again[n], want[n]), n


@pytest.mark.parametrize("width", [56, 512, 1000, 7168])
@pytest.mark.parametrize("value", [1.5, 1.75, 7.0])
def test_rows_of_one_value_have_its_exact_norm(width, value):
    # every partial sum of the squares is exact (a multiple of 2^-4 below 2^20), so their mean is value^2 and 1 / rms is
    # 1 / value rounded once
    x = torch.full((3, width), value, dtype=torch.bfloat16, device=DEV)
    one = torch.ones(width, dtype=torch.bfloat16, device=DEV)
    r = mok.add_rmsnorm(x, one, 0.0)
    assert torch.equal(r["rstd"].cpu(), torch.full((3,), value).reciprocal())
    # the gradient of a constant row through the norm is dy - mean(dy) times that: dy = 1 leaves only the roundings of
    # rstd (twice), of two products with it and of the one with sum, at most 5 * 2^-24 of 1 / value
    g = mok.add_rmsnorm_backward(torch.ones_like(x), r["sum"], one, r["rstd"])
    assert (g["dx"].abs() <= 2.0 ** -21 / value).all()


def ptr(t):
    return None if t is None else t.data_ptr()


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("name", list(TYPES))
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("p", [0.0, 0.25])
def test_forward_outputs_left_out(name, residual, p):
    x, w = randn((T, H), 11), (1.0 + 0.25 * randn((H,), 12).float()).to(torch.bfloat16)
    res = randn((T, H), 13, TYPES[name], 3.0) if residual else None
    rng = rng_state(3, 4) if p > 0 else None
    want = mok.add_rmsnorm(x, w, EPS, residual=res, p=p, rng=rng, stream_dtype=TYPES[name], mxfp8=True)
    shape = mok.mok_norm_shape(T, H, mok.MOK_STREAM_F32 if name == "fp32" else mok.MOK_STREAM_BF16, EPS, p)
    for keep in (("rstd", "y"), ("rstd", "y_elems", "y_scales"), ("rstd", "sum", "y")):
        o = {n: torch.full_like(want[n], 7) for n in keep}
        assert mok.mok_add_rmsnorm(shape, ptr(x), ptr(res), ptr(w), ptr(rng), ptr(o.get("sum")), ptr(o.get("y")),
                                   ptr(o.get("y_elems")), ptr(o.get("y_scales")), ptr(o["rstd"]), stream()) == mok.MOK_OK
        for n in keep:
            assert torch.equal(o[n], want[n]), (keep, n)


@pytest.mark.parametrize("name,p", [("bf16", 0.0), ("bf16", 0.25), ("fp32", 0.0), ("fp32", 0.25)])
@pytest.mark.parametrize("with_dsum", [False, True])
def test_backward_outputs_left_out(name, p, with_dsum):
    dy, s, w, rstd, dsum = backward_inputs(name)
    dsum = dsum if with_dsum else None
    rng = rng_state(5, 6) if p > 0 else None
    want = mok.add_rmsnorm_backward(dy, s, w, rstd, dsum=dsum, p=p, rng=rng)
    shape = mok.mok_norm_shape(T, H, mok.MOK_STREAM_F32 if name == "fp32" else mok.MOK_STREAM_BF16, 0.0, p)
    ws = torch.empty(T * H * 4, dtype=torch.uint8, device=DEV)
    for keep in (("dresidual", "dx"), ("dresidual",), ("dx",), ()):
        o = {n: torch.full_like(want[n], 7) for n in keep + ("dweight",)}
        assert mok.mok_add_rmsnorm_backward(shape, ptr(ws), ws.numel(), ptr(dy), ptr(s), ptr(w), ptr(rstd), ptr(dsum),
                                            ptr(rng), ptr(o.get("dresidual")), ptr(o.get("dx")), ptr(o["dweight"]),
                                            stream()) == mok.MOK_OK
        for n in o:
            assert torch.equal(o[n], want[n]), (keep, n)


def test_dropout_into_an_fp32_stream_without_a_residual():
    n, p = 8195, 0.25
    x, rng = randn((n,), 21), rng_state(7, 8)
    out = torch.full((n,), 7.0, device=DEV)
    assert mok.mok_dropout(ptr(x), None, n, p, ptr(rng), mok.MOK_STREAM_F32, ptr(out), stream()) == mok.MOK_OK
    assert torch.equal(out, mok.dropout(x, rng, p, residual=torch.zeros(n, device=DEV)))
