"""What the binding refuses around the routed experts, case by case and for the
reason it states. All tensors are on the CPU: the check of an argument comes
before the one for a GPU, whose message would answer any other call."""
import pytest
import torch

import mixture_experts_layer_table_amd as mok

P, FAR = 1 << 20, 1 << 44     # 16-byte aligned addresses that nothing reads, apart from each other


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _f32(*shape):
    return torch.zeros(shape)


@pytest.mark.parametrize("dx,message", [(_bf(4, 32), r"dx: shape \(4, 32\)"), (_f32(4, 64), "dx: dtype torch.float32"),
                                        (_bf(64, 4).T, "dx: must be contiguous")])
def test_norm_backward_checks_a_given_dx(dx, message):
    # bf16 stream and p == 0, where dx could also be left to dresidual
    grads = dict(dresidual=_bf(4, 64), dweight=_f32(64), dx=dx)
    with pytest.raises(ValueError, match=message):
        mok.add_rmsnorm_backward(_bf(4, 64), _bf(4, 64), _bf(64), _f32(4), grads=grads)


@pytest.mark.parametrize("n", [2 ** 37 - 8191, 2 ** 37, 2 ** 39])
def test_dropout_past_one_grid_is_refused(n):
    # 8,192 elements a workgroup of 256 threads: a grid of 2^32 threads cannot be launched
    a = [P + i * FAR for i in range(4)]
    assert mok.mok_dropout(a[0], a[1], n, 0.5, a[2], mok.MOK_STREAM_BF16, a[3], None) == mok.MOK_ERROR_INVALID_VALUE
    assert mok.mok_dropout_backward(a[0], n, 0.5, a[2], mok.MOK_STREAM_BF16, a[3], None) == \
        mok.MOK_ERROR_INVALID_VALUE


def _rng():
    return torch.zeros(2, dtype=torch.int64)


def _meta(t):
    return t.to("meta")


X = _bf(4, 64)
DROPOUT = [
    (dict(x=_f32(4, 64)), "x: dtype torch.float32"), (dict(x=_bf(64, 4).T), "x: must be contiguous"),
    (dict(rng=_rng().int()), "rng: dtype torch.int32"), (dict(rng=torch.zeros(3, dtype=torch.int64)), r"rng: shape \(3,\)"),
    (dict(rng=None), "rng: expected a torch.Tensor, got NoneType"), (dict(rng=_meta(_rng())), "rng: on meta"),
    (dict(p=1.0), "p: 1.0"), (dict(p=-0.5), "p: -0.5"), (dict(p=float("nan")), "p: nan"),
    (dict(residual=_bf(64, 4)), r"residual: shape \(64, 4\)"), (dict(residual=X.half()), "residual: dtype torch.float16"),
    (dict(residual=_meta(X)), "residual: on meta"), (dict(out=_f32(4, 64)), "out: dtype torch.float32"),
    (dict(residual=_f32(4, 64), out=X), "out: dtype torch.bfloat16"), (dict(out=_bf(4, 32)), r"out: shape \(4, 32\)"),
    (dict(), "must be on a GPU")]


@pytest.mark.parametrize("over,message", DROPOUT)
def test_dropout_refuses(over, message):
    with pytest.raises((ValueError, TypeError), match=message):
        mok.dropout(**dict(dict(x=X, rng=_rng(), p=0.1), **over))


@pytest.mark.parametrize("over,message", [
    (dict(dy=X.half()), "dy: dtype torch.float16"), (dict(dy=_bf(64, 4).T), "dy: must be contiguous"),
    (dict(rng=None), "rng: expected a torch.Tensor"), (dict(p=1.5), "p: 1.5"),
    (dict(dx=_f32(4, 64)), "dx: dtype torch.float32"), (dict(dx=_bf(256)), r"dx: shape \(256,\)"),
    (dict(), "must be on a GPU")])
def test_dropout_backward_refuses(over, message):
    with pytest.raises((ValueError, TypeError), match=message):
        mok.dropout_backward(**dict(dict(dy=X, rng=_rng(), p=0.1), **over))


def _outs(**over):
    o = dict(sum=_bf(4, 64), rstd=_f32(4), y=_bf(4, 64), y_elems=torch.zeros(4, 64, dtype=torch.uint8),
             y_scales=torch.zeros(4, 2, dtype=torch.uint8))
    return {n: t for n, t in dict(o, **over).items() if t is not None}


NORM = [
    (dict(x=_f32(4, 64)), "x: dtype torch.float32"), (dict(x=_bf(64)), r"x: shape \(64,\), expected \[T, H\]"),
    (dict(x=_bf(64, 4).T), "x: must be contiguous"), (dict(weight=_bf(32)), r"weight: shape \(32,\)"),
    (dict(weight=_f32(64)), "weight: dtype torch.float32"), (dict(weight=_meta(_bf(64))), "weight: on meta"),
    (dict(residual=_bf(4, 64), stream_dtype=torch.float32), "residual: dtype torch.bfloat16, expected torch.float32"),
    (dict(residual=_bf(5, 64)), r"residual: shape \(5, 64\)"), (dict(stream_dtype=torch.float16), "stream_dtype: dtype"),
    (dict(p=0.5), "rng: expected a torch.Tensor"), (dict(p=1.0, rng=_rng()), "p: 1.0"),
    (dict(y=False), "y and mxfp8 are both off"), (dict(x=_bf(4, 40), weight=_bf(40), mxfp8=True), "H = 40"),
    (dict(outs=_outs(sum=None)), "sum: expected a torch.Tensor"), (dict(outs=_outs(sum=_f32(4, 64))), "sum: dtype"),
    (dict(outs=_outs(rstd=_f32(3))), r"rstd: shape \(3,\)"), (dict(outs=_outs(y=_bf(4, 32))), r"y: shape \(4, 32\)"),
    (dict(outs=_outs(y=None)), "y: expected a torch.Tensor"),
    (dict(mxfp8=True, outs=_outs(y_elems=_bf(4, 64))), "y_elems: dtype torch.bfloat16"),
    (dict(mxfp8=True, outs=_outs(y_scales=torch.zeros(4, 1, dtype=torch.uint8))), r"y_scales: shape \(4, 1\)"),
    (dict(), "must be on a GPU")]


@pytest.mark.parametrize("over,message", NORM)
def test_norm_refuses(over, message):
    with pytest.raises((ValueError, TypeError), match=message):
        mok.add_rmsnorm(**dict(dict(x=X, weight=_bf(64), eps=1e-6), **over))


@pytest.mark.parametrize("over,message", [
    (dict(sum=X.half()), "sum: dtype torch.float16"), (dict(sum=_bf(64)), r"sum: shape \(64,\), expected \[T, H\]"),
    (dict(dy=_f32(4, 64)), "dy: dtype torch.float32"), (dict(dy=_bf(3, 64)), r"dy: shape \(3, 64\)"),
    (dict(weight=_bf(8)), r"weight: shape \(8,\)"), (dict(rstd=_f32(3)), r"rstd: shape \(3,\)"),
    (dict(rstd=_bf(4)), "rstd: dtype torch.bfloat16"), (dict(dsum=_f32(4, 64)), "dsum: dtype torch.float32"),
    (dict(sum=_f32(4, 64), dsum=X), "dsum: dtype torch.bfloat16"), (dict(p=0.5), "rng: expected a torch.Tensor"),
    (dict(grads=dict(dweight=_f32(64))), "dresidual: expected a torch.Tensor"),
    (dict(grads=dict(dresidual=X, dweight=_bf(64))), "dweight: dtype torch.bfloat16"),
    (dict(sum=_f32(4, 64), grads=dict(dresidual=_f32(4, 64), dweight=_f32(64))), "dx: expected a torch.Tensor"),
    (dict(), "must be on a GPU")])
def test_norm_backward_refuses(over, message):
    with pytest.raises((ValueError, TypeError), match=message):
        mok.add_rmsnorm_backward(**dict(dict(dy=X, sum=_bf(4, 64), weight=_bf(64), rstd=_f32(4)), **over))


def _u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def _codes(rows, K):
    return _u8(rows, K), _u8(rows, K // 32)


WS = mok.get_ffn_workspace(mok.MOK_BF16, device="cpu", num_tokens=8, hidden_size=128, intermediate_size=64)
W = mok.weights_bf16(_bf(128, 64), _bf(1, 128, 64), _bf(64, 128))
WS_MX = mok.get_ffn_workspace(mok.MOK_MXFP8, device="cpu", num_tokens=8, hidden_size=256, intermediate_size=128)
FWD = mok.weights_mxfp8(_codes(128, 256), _codes(128, 256), _codes(256, 128), "fwd")
BWD = mok.weights_mxfp8(_codes(256, 128), _codes(256, 128), _codes(128, 256), "bwd")
ROWS = _bf(8, 128)


def _w(gate=(128, 64), up=(128, 64), down=(64, 128)):
    return mok.weights_bf16(_bf(*gate), _bf(*up), _bf(*down))


@pytest.mark.parametrize("ws,x,w,over,message", [
    (WS, _bf(9, 128), W, {}, r"x: shape \(9, 128\), expected \[T, 128\] with T <= 8"),
    (WS, _bf(8, 64), W, {}, r"x: shape \(8, 64\)"), (WS, _f32(8, 128), W, {}, "x: dtype torch.float32"),
    (WS, _bf(128, 8).T, W, {}, "x: must be contiguous"), (WS, _meta(ROWS), W, {}, "x: on meta"),
    (WS, ROWS, _w(gate=(64, 128)), {}, r"w_gate: shape \(64, 128\)"), (WS, ROWS, _w(up=(2, 128, 64)), {}, "w_up: shape"),
    (WS, ROWS, _w(down=(128, 64)), {}, "w_down: shape"), (WS, ROWS, FWD, {}, "BF16 mode needs bf16 weights"),
    (WS, ROWS, mok.weights_bf16(_f32(128, 64), _bf(128, 64), _bf(64, 128)), {}, "w_gate: dtype torch.float32"),
    (WS, ROWS, W, dict(addend=_bf(8, 64)), r"addend: shape \(8, 64\)"),
    (WS, ROWS, W, dict(addend=_f32(8, 128)), "addend: dtype"), (WS, ROWS, W, dict(out=_bf(7, 128)), r"out: shape \(7, 128\)"),
    (WS, ROWS, W, dict(h=_bf(8, 64)), r"h: shape \(8, 64\)"), (WS, ROWS, W, {}, "must be on a GPU"),
    (WS_MX, _bf(8, 256), FWD, {}, r"MXFP8 mode takes \(elems, scales\)"),
    (WS_MX, (_u8(8, 128), _u8(8, 4)), FWD, {}, r"x elements: shape \(8, 128\)"),
    (WS_MX, (_u8(8, 256), _u8(8, 4)), FWD, {}, r"x scales: shape \(8, 4\)"),
    (WS_MX, (_bf(8, 256), _u8(8, 8)), FWD, {}, "x elements: dtype torch.bfloat16"),
    (WS_MX, _codes(8, 256), W, {}, "MXFP8 mode needs quantized weights"),
    (WS_MX, _codes(8, 256), BWD, {}, "quantized for bwd, used in fwd"),
    (WS_MX, _codes(8, 256), mok.weights_mxfp8(_codes(128, 256), _codes(256, 128), _codes(256, 128)), {},
     "up elements: shape"),
    (WS_MX, _codes(8, 256), mok.weights_mxfp8(_codes(128, 256), _codes(128, 256), (_u8(256, 128), _u8(256, 2))), {},
     "down scales: shape"),
    (WS_MX, _codes(8, 256), FWD, {}, "must be on a GPU")])
def test_ffn_forward_refuses(ws, x, w, over, message):
    with pytest.raises(ValueError, match=message):
        mok.ffn_forward(ws, x, w, **over)


def _grads(**over):
    return dict(dict(dx=_bf(8, 128), dw_gate=_bf(128, 64), dw_up=_bf(128, 64), dw_down=_bf(64, 128)), **over)


@pytest.mark.parametrize("over,message", [
    (dict(x=_bf(9, 128)), r"x: shape \(9, 128\)"), (dict(x=_f32(8, 128)), "x: dtype"),
    (dict(h=_bf(8, 64)), r"h: shape \(8, 64\), expected \(8, 128\)"), (dict(dy=_bf(4, 128)), r"dy: shape \(4, 128\)"),
    (dict(dy=_f32(8, 128)), "dy: dtype"), (dict(addend=_bf(8, 64)), "addend: shape"),
    (dict(weights=_w(down=(128, 64))), "w_down: shape"), (dict(weights=BWD), "BF16 mode needs bf16 weights"),
    (dict(ws=WS_MX, x=_bf(8, 256), dy=_bf(8, 256), h=_bf(8, 256), weights=FWD), "quantized for fwd, used in bwd"),
    (dict(grads=_grads(dw_up=_f32(128, 64))), "dw_up: dtype"), (dict(grads=_grads(dw_down=_bf(128, 64))), "dw_down: shape"),
    (dict(grads=_grads(dx=None)), "dx: expected a torch.Tensor"), (dict(), "must be on a GPU")])
def test_ffn_backward_refuses(over, message):
    with pytest.raises((ValueError, TypeError), match=message):
        mok.ffn_backward(**dict(dict(ws=WS, x=ROWS, weights=W, h=_bf(8, 128), dy=_bf(8, 128)), **over))


@pytest.mark.parametrize("shape", [dict(hidden_size=100), dict(intermediate_size=32), dict(num_tokens=-1)])
def test_workspace_refuses(shape):
    with pytest.raises(mok.MokError, match="mok_ffn_query_size: MOK_ERROR_INVALID_VALUE"):
        mok.get_ffn_workspace(mok.MOK_BF16, device="cpu",
                              **dict(dict(num_tokens=8, hidden_size=128, intermediate_size=64), **shape))
