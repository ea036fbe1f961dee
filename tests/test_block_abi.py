"""Refusals and sizes of the operators around the routed experts: every bad
argument is answered on the host, before anything is enqueued (no GPU here:
an accepted call would fail to launch and say so with another status)."""
import ctypes

import pytest
import torch

import mixture_experts_layer_table_amd as mok

BAD = mok.MOK_ERROR_INVALID_VALUE
P = 1 << 20          # a 16-byte aligned address that nothing reads
FAR = 1 << 44        # spacing that keeps fake buffers apart


def _a(i):
    return P + i * FAR


# ------------------------------------------------------------------------- dropout

def _dropout(**over):
    k = dict(x=_a(0), residual=_a(1), n=100, p=0.5, rng=_a(2), dtype=mok.MOK_STREAM_BF16, out=_a(3))
    k.update(over)
    return mok.mok_dropout(k["x"], k["residual"], k["n"], k["p"], k["rng"], k["dtype"], k["out"], None)


@pytest.mark.parametrize("over", [dict(n=-1), dict(n=1 << 40), dict(p=1.0), dict(p=-0.1), dict(p=float("nan")),
                                  dict(rng=None), dict(rng=_a(2) + 4), dict(dtype=2), dict(dtype=-1), dict(x=None),
                                  dict(x=_a(0) + 2), dict(residual=_a(1) + 8), dict(out=None), dict(out=_a(3) + 1),
                                  dict(out=_a(0) + 16), dict(out=_a(1) - 16), dict(out=_a(2)), dict(out=_a(2) - 192),
                                  dict(dtype=mok.MOK_STREAM_F32, out=_a(0))])   # fp32 rows over the bf16 branch
def test_dropout_refuses(over):
    assert _dropout(**over) == BAD


def test_dropout_of_nothing_is_a_no_op():
    assert _dropout(n=0, x=None, residual=None, out=None, p=0.0, rng=None) == mok.MOK_OK


@pytest.mark.parametrize("over", [dict(n=-1), dict(p=1.0), dict(rng=None), dict(dtype=3), dict(dy=None), dict(dx=None),
                                  dict(dx=_a(0) + 32), dict(dx=_a(2)), dict(dtype=mok.MOK_STREAM_F32, dx=_a(0))])
def test_dropout_backward_refuses(over):
    k = dict(dy=_a(0), n=100, p=0.5, rng=_a(2), dtype=mok.MOK_STREAM_BF16, dx=_a(3))
    k.update(over)
    assert mok.mok_dropout_backward(k["dy"], k["n"], k["p"], k["rng"], k["dtype"], k["dx"], None) == BAD


# ------------------------------------------------------------------------- norm

def _norm(shape=None, **over):
    s = dict(T=8, H=64, stream_dtype=0, eps=1e-6, p=0.0)
    s.update(shape or {})
    k = dict(x=_a(0), residual=_a(1), weight=_a(2), rng=None, sum=_a(3), y=_a(4), elems=_a(5), scales=_a(6), rstd=_a(7))
    k.update(over)
    return mok.mok_add_rmsnorm(mok.mok_norm_shape(**s), *k.values(), None)


@pytest.mark.parametrize("shape", [dict(T=-1), dict(T=1 << 31), dict(H=0), dict(H=68), dict(H=16392),
                                   dict(H=40),                                   # MXFP8 rows: no whole 32-blocks
                                   dict(stream_dtype=2), dict(eps=-1.0), dict(eps=float("nan")),
                                   dict(eps=float("inf")), dict(p=1.0), dict(p=-0.5), dict(p=0.5)])  # p without rng
def test_norm_refuses_shapes(shape):
    assert _norm(shape) == BAD


@pytest.mark.parametrize("over", [dict(x=None), dict(weight=None), dict(rstd=None), dict(rstd=_a(7) + 2),
                                  dict(y=None, elems=None, scales=None), dict(elems=None), dict(scales=None),
                                  dict(x=_a(0) + 8), dict(sum=_a(3) + 4), dict(y=_a(0)), dict(y=_a(3)),
                                  dict(sum=_a(1) + 128), dict(sum=_a(2)), dict(rstd=_a(2)), dict(elems=_a(1)),
                                  dict(scales=_a(5))])
def test_norm_refuses_buffers(over):
    assert _norm(**over) == BAD


def test_norm_of_no_rows_is_a_no_op():
    assert mok.mok_add_rmsnorm(mok.mok_norm_shape(0, 64, 0, 1e-6, 0.0), None, None, None, None, None, _a(0), None, None,
                               None, None) == mok.MOK_OK


def _norm_bwd(shape=None, **over):
    s = dict(T=8, H=64, stream_dtype=0, eps=1e-6, p=0.0)
    s.update(shape or {})
    k = dict(ws=_a(0), ws_bytes=1 << 30, dy=_a(1), sum=_a(2), weight=_a(3), rstd=_a(4), dsum=_a(5), rng=None,
             dres=_a(6), dx=_a(7), dweight=_a(8))
    k.update(over)
    return mok.mok_add_rmsnorm_backward(mok.mok_norm_shape(**s), *k.values(), None)


@pytest.mark.parametrize("over", [dict(ws=None), dict(dy=None), dict(sum=None), dict(weight=None), dict(rstd=None),
                                  dict(dweight=None), dict(dweight=_a(8) + 4), dict(dres=_a(2)), dict(dres=_a(1)),
                                  dict(dres=_a(5) + 16), dict(dx=_a(6)), dict(dx=_a(1) + 16), dict(dx=_a(5)),
                                  dict(dweight=_a(3)), dict(ws=_a(2))])
def test_norm_backward_refuses_buffers(over):
    assert _norm_bwd(**over) == BAD


def test_norm_backward_refuses_shapes_and_small_workspaces():
    for shape in (dict(T=-1), dict(H=12), dict(H=16392), dict(stream_dtype=7), dict(p=0.5)):
        assert _norm_bwd(shape) == BAD
    need = ctypes.c_size_t()
    sizes = []
    for T in (0, 1, 8, 777, 16384, 100000):
        assert mok.mok_add_rmsnorm_backward_size(mok.mok_norm_shape(T, 64, 0, 0.0, 0.0), ctypes.byref(need)) == 0
        sizes.append(need.value)
    assert sizes == sorted(sizes)         # a workspace for T rows serves fewer
    assert _norm_bwd(dict(T=777), ws_bytes=sizes[3] - 1) == mok.MOK_ERROR_BUFFER_TOO_SMALL
    assert mok.mok_add_rmsnorm_backward_size(mok.mok_norm_shape(8, 64, 0, 0.0, 0.0), None) == BAD


# ------------------------------------------------------------------------- feed-forward block

BAD_FFN = [dict(T=-1), dict(H=0), dict(I=0), dict(H=96), dict(I=32), dict(precision=mok.MOK_MXFP8, H=192),
           dict(precision=mok.MOK_MXFP8, I=64), dict(precision=mok.MOK_MXFP8_WGRAD), dict(precision=9),
           dict(T=1 << 17, H=8192), dict(T=1 << 19, I=1024), dict(H=32768, I=32704), dict(H=32704, I=32768),
           dict(T=1, H=64, I=(1 << 20) + 64), dict(T=1, H=(1 << 20) + 64, I=64)]


@pytest.mark.parametrize("over", BAD_FFN)
def test_ffn_refuses_shapes(over):
    s = dict(T=64, H=128, I=128, precision=mok.MOK_BF16)
    s.update(over)
    need = ctypes.c_size_t()
    assert mok.mok_ffn_query_size(mok.mok_ffn_shape(**s), ctypes.byref(need)) == BAD


@pytest.mark.parametrize("shape", [
    (1, 64, 1 << 20, 0), (1, 1 << 20, 64, 0), (1, 128, 1 << 20, 1), ((1 << 23) - 1, 64, 64, 0)])
def test_ffn_shapes_at_the_bounds_accepted(shape):
    need = ctypes.c_size_t()
    assert mok.mok_ffn_query_size(mok.mok_ffn_shape(*shape), ctypes.byref(need)) == mok.MOK_OK and need.value > 0


@pytest.mark.parametrize("precision", [mok.MOK_BF16, mok.MOK_MXFP8])
def test_ffn_workspace_serves_fewer_rows(precision):
    need, last = ctypes.c_size_t(), 0
    for T in (0, 1, 2, 31, 32, 33, 100, 128, 129, 500, 777, 1000, 1001, 2047, 2048, 4000, 16384):
        assert mok.mok_ffn_query_size(mok.mok_ffn_shape(T, 7168, 2048, precision), ctypes.byref(need)) == 0
        assert need.value >= last
        last = need.value


def _weights(mx):
    w = [_a(20 + i) for i in range(6)]
    return mok.mok_weights(None, None, None, *w) if mx else mok.mok_weights(*w[:3])


def _ffn(mx, **over):
    k = dict(ws=_a(0), ws_bytes=1 << 40, x=None if mx else _a(1), elems=_a(2) if mx else None,
             scales=_a(3) if mx else None, w=_weights(mx), addend=_a(4), out=_a(5), h=_a(6))
    T = over.pop("T", 64)
    k.update(over)
    return mok.mok_ffn_forward(mok.mok_ffn_shape(T, 128, 128, int(mx)), *k.values(), None)


@pytest.mark.parametrize("mx,over", [(False, dict(ws=None)), (False, dict(x=None)), (False, dict(x=_a(1) + 2)),
                                     (False, dict(out=None)), (False, dict(h=_a(6) + 8)), (False, dict(out=_a(1))),
                                     (False, dict(out=_a(4) + 16)), (False, dict(h=_a(4))), (False, dict(h=_a(5))),
                                     (False, dict(out=_a(20))), (False, dict(ws=_a(1))), (True, dict(elems=None)),
                                     (True, dict(scales=None)), (True, dict(elems=_a(2) + 4)), (True, dict(out=_a(2))),
                                     (False, dict(w=mok.mok_weights(_a(20), _a(21), None))),
                                     (True, dict(w=mok.mok_weights(_a(20), _a(21), _a(22))))])
def test_ffn_forward_refuses(mx, over):
    assert _ffn(mx, **over) == BAD


def test_ffn_small_workspace_and_no_rows():
    need = ctypes.c_size_t()
    mok.mok_ffn_query_size(mok.mok_ffn_shape(64, 128, 128, 0), ctypes.byref(need))
    assert _ffn(False, ws_bytes=need.value - 1) == mok.MOK_ERROR_BUFFER_TOO_SMALL
    assert _ffn(False, T=0, x=None, addend=None, out=None, h=None) == mok.MOK_OK


@pytest.mark.parametrize("over", [dict(ws=None), dict(x=None), dict(h=None), dict(dy=None), dict(dx=None),
                                  dict(dw_gate=None), dict(dw_up=None), dict(dw_down=_a(9) + 2), dict(dx=_a(3)),
                                  dict(dx=_a(1)), dict(dx=_a(4) + 64), dict(dw_gate=_a(4)), dict(dw_up=_a(6)),
                                  dict(dw_down=_a(2)), dict(dw_gate=_a(20))])
def test_ffn_backward_refuses(over):
    k = dict(ws=_a(0), ws_bytes=1 << 40, x=_a(1), w=_weights(False), h=_a(2), dy=_a(3), addend=_a(4), dx=_a(5),
             dw_gate=_a(6), dw_up=_a(7), dw_down=_a(8))
    k.update(over)
    assert mok.mok_ffn_backward(mok.mok_ffn_shape(64, 128, 128, 0), *k.values(), None) == BAD


# ------------------------------------------------------------------------- binding

def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_binding_refuses_wrong_tensors():
    rng = torch.zeros(2, dtype=torch.int64)
    for bad in (lambda: mok.dropout(_bf(4, 8).float(), rng, 0.1),                       # branch must be bf16
                lambda: mok.dropout(_bf(8, 4).T, rng, 0.1),                             # not contiguous
                lambda: mok.dropout(_bf(4, 8), rng.int(), 0.1),
                lambda: mok.dropout(_bf(4, 8), rng, 1.0),
                lambda: mok.dropout(_bf(4, 8), rng, 0.1, residual=_bf(8, 4)),
                lambda: mok.dropout(_bf(4, 8), rng, 0.1, residual=_bf(4, 8).half()),
                lambda: mok.dropout(_bf(4, 8), rng, 0.1),                               # not on a GPU
                lambda: mok.dropout_backward(_bf(4, 8).half(), rng, 0.1),
                lambda: mok.add_rmsnorm(_bf(4, 64), _bf(32), 1e-6),
                lambda: mok.add_rmsnorm(_bf(64), _bf(64), 1e-6),
                lambda: mok.add_rmsnorm(_bf(4, 40), _bf(40), 1e-6, mxfp8=True),
                lambda: mok.add_rmsnorm(_bf(4, 64), _bf(64), 1e-6, residual=_bf(4, 64), stream_dtype=torch.float32),
                lambda: mok.add_rmsnorm_backward(_bf(4, 64), _bf(4, 64), _bf(64), torch.zeros(3)),
                lambda: mok.add_rmsnorm_backward(_bf(4, 64), _bf(4, 64).float(), _bf(64), torch.zeros(4),
                                                 dsum=_bf(4, 64))):
        with pytest.raises((ValueError, TypeError)):
            bad()


def test_binding_checks_the_block():
    ws = mok.get_ffn_workspace(mok.MOK_BF16, device="cpu", num_tokens=8, hidden_size=128, intermediate_size=64)
    w = mok.weights_bf16(_bf(128, 64), _bf(1, 128, 64), _bf(64, 128))
    wm = mok.get_ffn_workspace(mok.MOK_MXFP8, device="cpu", num_tokens=8, hidden_size=128, intermediate_size=128)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    q = lambda r, k: (u8(r, k), u8(r, k // 32))  # noqa: E731
    fwd = mok.weights_mxfp8(q(128, 128), q(128, 128), q(128, 128), "fwd")
    for bad in (lambda: mok.ffn_forward(ws, _bf(9, 128), w),                            # more rows than the workspace
                lambda: mok.ffn_forward(ws, _bf(8, 64), w),
                lambda: mok.ffn_forward(ws, _bf(8, 128), mok.weights_bf16(_bf(64, 128), _bf(128, 64), _bf(64, 128))),
                lambda: mok.ffn_forward(ws, _bf(8, 128), fwd),
                lambda: mok.ffn_forward(ws, _bf(8, 128), w, addend=_bf(8, 64)),
                lambda: mok.ffn_forward(wm, _bf(8, 128), fwd),                          # MXFP8 takes quantized rows
                lambda: mok.ffn_forward(wm, (u8(8, 128), u8(8, 3)), fwd),
                lambda: mok.ffn_backward(wm, _bf(8, 128), fwd, _bf(8, 256), _bf(8, 128)),   # forward's orientation
                lambda: mok.ffn_backward(ws, _bf(8, 128), w, _bf(8, 64), _bf(8, 128)),
                lambda: mok.ffn_forward(ws, _bf(8, 128), w)):                           # not on a GPU
        with pytest.raises((ValueError, TypeError)):
            bad()
    with pytest.raises(mok.MokError):
        mok.get_ffn_workspace(mok.MOK_BF16, device="cpu", num_tokens=8, hidden_size=100, intermediate_size=64)
