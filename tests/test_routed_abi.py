"""Refusals, sizes and limits of the routed experts' parts, at the C ABI and in the
binding: every bad argument is answered on the host, before anything is enqueued."""
import ctypes

import pytest
import torch

import mixture_experts_layer_table_amd as mok
import routed_reference as R

BAD, SMALL, UNSUPPORTED = mok.MOK_ERROR_INVALID_VALUE, mok.MOK_ERROR_BUFFER_TOO_SMALL, mok.MOK_ERROR_UNSUPPORTED
P, FAR = 1 << 20, 1 << 44     # 16-byte aligned addresses that nothing reads, apart from each other


def _a(i):
    return P + i * FAR


# ------------------------------------------------------------------------- sort

@pytest.mark.parametrize("T,k,E,align", [(0, 1, 1, 1), (1, 8, 256, 16), (2048, 8, 256, 128), (163840, 1, 8, 128),
                                         (5, 3, 4096, 1024), (1 << 20, 8, 64, 1)])
def test_sort_sizes(T, k, E, align):
    rows, need = ctypes.c_int64(), ctypes.c_size_t()
    s = mok.mok_sort_shape(T, k, E, align)
    assert mok.mok_sort_tokens_size(s, ctypes.byref(rows), ctypes.byref(need)) == mok.MOK_OK
    assert rows.value == R.sort_rows(T * k, E, align) == mok.sort_rows(T, k, E, align)
    assert need.value == 0 or T * k > 32768 or E > 512     # one launch takes no workspace
    assert mok.mok_sort_tokens_size(s, None, None) == mok.MOK_OK


BAD_SORT = [dict(T=-1), dict(T=1 << 31), dict(k=0), dict(E=0), dict(E=4097), dict(align=0), dict(align=1025),
            dict(T=1 << 30, k=2), dict(T=(1 << 30) - 1, k=2, E=4096, align=1024)]


@pytest.mark.parametrize("over", BAD_SORT)
def test_sort_refuses_shapes(over):
    s = mok.mok_sort_shape(**{**dict(T=8, k=2, E=4, align=16), **over})
    assert mok.mok_sort_tokens_size(s, None, None) == BAD
    assert mok.mok_sort_tokens(s, _a(0), 1 << 40, _a(1), _a(2), _a(3), _a(4), None) == BAD


@pytest.mark.parametrize("over", [dict(ids=None), dict(offsets=None), dict(slots=None), dict(row_slots=None), dict(ids=_a(1) + 4), dict(slots=_a(1)), dict(row_slots=_a(3)),
                                  dict(offsets=_a(3)), dict(row_slots=_a(1) - 16)])
def test_sort_refuses_buffers(over):
    k = {**dict(ws=_a(0), n=1 << 20, ids=_a(1), offsets=_a(2), slots=_a(3), row_slots=_a(4)), **over}
    assert mok.mok_sort_tokens(mok.mok_sort_shape(8, 2, 4, 16), *k.values(), None) == BAD


def test_sort_refuses_a_small_workspace():
    s, need = mok.mok_sort_shape(1 << 16, 1, 8, 1), ctypes.c_size_t()
    mok.mok_sort_tokens_size(s, None, ctypes.byref(need))
    assert need.value > 0
    assert mok.mok_sort_tokens(s, _a(0), need.value - 1, _a(1), _a(2), _a(3), _a(4), None) == SMALL
    assert mok.mok_sort_tokens(s, None, need.value, _a(1), _a(2), _a(3), _a(4), None) == BAD


# ------------------------------------------------------------------------- rows

def _shape(**over):
    return mok.mok_rows_shape(**{**dict(T=8, rows=40, k=2, E=4, H=64, dtype=0), **over})


BAD_ROWS = [dict(T=-1), dict(T=1 << 31), dict(rows=-1), dict(rows=1 << 31), dict(k=0), dict(E=0), dict(E=4097),
            dict(H=0), dict(H=60), dict(H=(1 << 20) + 8), dict(dtype=2), dict(T=1 << 30, k=2)]


def _permute(shape=None, **over):
    k = dict(x=_a(0), offsets=_a(1), slots=_a(2), row_slots=_a(3), rows=_a(4), elems=_a(5), scales=_a(6))
    k.update(over)
    return mok.mok_permute(_shape(**(shape or {})), *k.values(), None)


def _unpermute(shape=None, **over):
    k = dict(y=_a(0), slots=_a(1), w=_a(2), addend=_a(3), out=_a(4))
    k.update(over)
    return mok.mok_unpermute(_shape(**(shape or {})), *k.values(), None)


def _unpermute_bwd(shape=None, **over):
    k = dict(dout=_a(0), y=_a(1), offsets=_a(2), slots=_a(3), row_slots=_a(4), w=_a(5), dy=_a(6), dw=_a(7))
    k.update(over)
    return mok.mok_unpermute_backward(_shape(**(shape or {})), *k.values(), None)


@pytest.mark.parametrize("shape", BAD_ROWS)
def test_rows_refuse_shapes(shape):
    assert _permute(shape) == BAD and _unpermute(shape) == BAD and _unpermute_bwd(shape) == BAD
    assert mok.mok_permute_backward(_shape(**shape), _a(0), _a(1), _a(2), None) == BAD


@pytest.mark.parametrize("over", [dict(x=None), dict(offsets=None), dict(slots=None), dict(row_slots=None),
                                  dict(rows=None, elems=None, scales=None), dict(elems=None), dict(scales=None),
                                  dict(x=_a(0) + 8), dict(rows=_a(4) + 4), dict(rows=_a(0)), dict(elems=_a(4)),
                                  dict(scales=_a(2)), dict(elems=_a(3) + 16)])
def test_permute_refuses_buffers(over):
    assert _permute(**over) == BAD


def test_permute_refuses_quantized_rows_of_odd_width():
    assert _permute(dict(H=72)) == BAD


@pytest.mark.parametrize("over", [dict(y=None), dict(slots=None), dict(out=None), dict(w=_a(2) + 4), dict(out=_a(0)),
                                  dict(out=_a(3) + 16), dict(out=_a(1)), dict(out=_a(2)), dict(addend=_a(3) + 2)])
def test_unpermute_refuses_buffers(over):
    assert _unpermute(**over) == BAD


@pytest.mark.parametrize("over", [dict(drows=None), dict(slots=None), dict(dx=None), dict(dx=_a(0)), dict(dx=_a(1))])
def test_permute_backward_refuses_buffers(over):
    k = {**dict(drows=_a(0), slots=_a(1), dx=_a(2)), **over}
    assert mok.mok_permute_backward(_shape(), *k.values(), None) == BAD


@pytest.mark.parametrize("over", [dict(dout=None), dict(y=None), dict(offsets=None), dict(slots=None),
                                  dict(row_slots=None), dict(w=None), dict(dy=None), dict(dw=None), dict(dy=_a(0)),
                                  dict(dy=_a(1) + 16), dict(dw=_a(1)), dict(dw=_a(5)), dict(dw=_a(6)), dict(dy=_a(2))])
def test_unpermute_backward_refuses_buffers(over):
    assert _unpermute_bwd(**over) == BAD


def test_rows_of_nothing_are_no_ops():
    empty = dict(T=0, rows=0)
    assert _permute(empty, **{n: None for n in ("x", "offsets", "slots", "row_slots", "rows", "elems", "scales")}) == 0
    assert _unpermute(empty, **{n: None for n in ("y", "slots", "w", "addend", "out")}) == 0
    assert _unpermute_bwd(empty, **{n: None for n in ("dout", "y", "offsets", "slots", "row_slots", "w", "dy", "dw")}) == 0


# ------------------------------------------------------------------------- blocks of 128

def _quantize(**over):
    k = dict(src=_a(0), dtype=0, batch=2, rows=40, K=64, flags=0, elems=_a(1), scales=_a(2))
    k.update(over)
    return mok.mok_fp8_quantize(*k.values(), None)


@pytest.mark.parametrize("over", [dict(src=None), dict(elems=None), dict(scales=None), dict(dtype=2), dict(batch=-1),
                                  dict(batch=65536), dict(rows=-1), dict(rows=1 << 31), dict(K=-16), dict(K=40),
                                  dict(K=1 << 31), dict(rows=1 << 24, K=1 << 16), dict(flags=8), dict(flags=1, rows=36),
                                  dict(flags=mok.MOK_FP8_GLU | mok.MOK_FP8_TILE), dict(flags=mok.MOK_FP8_GLU, dtype=1),
                                  dict(src=_a(0) + 2), dict(elems=_a(0)), dict(scales=_a(0) + 64), dict(scales=_a(1)),
                                  dict(flags=mok.MOK_FP8_GLU, elems=_a(0) + 2 * 2 * 40 * 64 * 2 - 16)])
def test_quantize_refuses(over):
    assert _quantize(**over) == BAD


def test_quantize_of_nothing_is_a_no_op():
    assert _quantize(rows=0, src=None, elems=None, scales=None) == mok.MOK_OK


@pytest.mark.parametrize("over", [dict(da=None), dict(h=None), dict(dh=None), dict(T=-1), dict(T=1 << 31), dict(I=0),
                                  dict(I=12), dict(dh=_a(0)), dict(dh=_a(1) + 16), dict(h=_a(1) + 8)])
def test_glu_backward_refuses(over):
    k = {**dict(da=_a(0), h=_a(1), T=8, I=64, dh=_a(2)), **over}
    assert mok.mok_glu_backward(*k.values(), None) == BAD


def _fp8(**over):
    return mok.mok_fp8_shape(**{**dict(M=32, N=64, K=256, E=0, out_dtype=0), **over})


BAD_FP8 = [dict(M=-1), dict(N=0), dict(N=40), dict(N=(1 << 20) + 16), dict(K=0), dict(K=24), dict(K=(1 << 20) + 16),
           dict(E=-1), dict(E=4097), dict(out_dtype=2)]


@pytest.mark.parametrize("over", BAD_FP8)
def test_products_refuse_shapes(over):
    need = ctypes.c_size_t()
    assert mok.mok_fp8_matmul_size(_fp8(**over), ctypes.byref(need)) == BAD
    assert mok.mok_fp8_wgrad_size(_fp8(**over), ctypes.byref(need)) == BAD
    assert mok.mok_fp8_matmul(_fp8(**over), _a(0), 1 << 40, _a(1), _a(2), _a(3), _a(4), None, _a(5), None) == BAD
    assert mok.mok_fp8_wgrad(_fp8(**over), _a(0), 1 << 40, _a(1), _a(2), _a(3), _a(4), None, None, _a(5), None) == BAD


def test_product_limits():
    need = ctypes.c_size_t()
    assert mok.mok_fp8_matmul_size(_fp8(M=1 << 31), ctypes.byref(need)) == BAD
    assert mok.mok_fp8_wgrad_size(_fp8(M=1 << 23), ctypes.byref(need)) == BAD
    assert mok.mok_fp8_wgrad_size(_fp8(M=24), ctypes.byref(need)) == BAD
    assert mok.mok_fp8_matmul_size(_fp8(M=(1 << 31) - 1, N=1 << 20), ctypes.byref(need)) == UNSUPPORTED
    assert mok.mok_fp8_wgrad_size(_fp8(N=1 << 20, K=1 << 20), ctypes.byref(need)) == UNSUPPORTED
    assert mok.mok_fp8_matmul_size(_fp8(), None) == BAD and mok.mok_fp8_wgrad_size(_fp8(), None) == BAD


def _matmul(shape=None, **over):
    k = dict(ws=_a(0), n=1 << 40, a=_a(1), asc=_a(2), b=_a(3), bsc=_a(4), offsets=None, out=_a(5))
    k.update(over)
    return mok.mok_fp8_matmul(_fp8(**(shape or {})), *k.values(), None)


@pytest.mark.parametrize("over", [dict(a=None), dict(asc=None), dict(b=None), dict(bsc=None),
                                  dict(out=None), dict(offsets=_a(6)), dict(a=_a(1) + 8), dict(out=_a(1)),
                                  dict(out=_a(3) + 16), dict(out=_a(2)), dict(out=_a(4))])
def test_matmul_refuses_buffers(over):
    assert _matmul(**over) == BAD


def test_matmul_refuses_missing_offsets_and_small_workspaces():
    assert _matmul(dict(E=2)) == BAD
    assert _matmul(dict(E=2), offsets=_a(5)) == BAD          # the output's buffer
    runs = dict(M=128, N=2064, K=7168)                       # a contraction in runs: with a workspace
    assert _matmul(runs, n=0) == SMALL
    for ws in (None, _a(0) + 8, _a(1), _a(3), _a(5)):
        assert _matmul(runs, ws=ws) == BAD
    assert _matmul(dict(M=0), a=None, asc=None, out=None) == mok.MOK_OK


def _wgrad(shape=None, **over):
    k = dict(ws=_a(0), n=1 << 40, dy=_a(1), dysc=_a(2), x=_a(3), xsc=_a(4), offsets=None, addend=_a(6), out=_a(5))
    k.update(over)
    return mok.mok_fp8_wgrad(_fp8(**(shape or {})), *k.values(), None)


@pytest.mark.parametrize("over", [dict(dy=None), dict(dysc=None), dict(x=None), dict(xsc=None),
                                  dict(out=None), dict(offsets=_a(7)), dict(addend=_a(6) + 2), dict(out=_a(1)),
                                  dict(out=_a(6) + 16), dict(out=_a(3))])
def test_wgrad_refuses_buffers(over):
    assert _wgrad(**over) == BAD


def test_wgrad_refuses_missing_offsets_and_small_workspaces():
    assert _wgrad(dict(E=3)) == BAD
    runs = dict(M=8192, N=512, K=512)                        # a contraction in runs: with a workspace
    assert _wgrad(runs, n=0) == SMALL
    for ws in (None, _a(0) + 8, _a(1), _a(4), _a(5), _a(6)):
        assert _wgrad(runs, ws=ws) == BAD


# ------------------------------------------------------------------------- the binding

def _i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _f32(*shape):
    return torch.zeros(shape)


def _u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


SORT = dict(offsets=_i32(5), slots=_i32(8, 2), row_slots=_i32(40))
CODES, TILES = (_u8(32, 256), _f32(2, 32)), (_u8(64, 256), _f32(1, 2))


@pytest.mark.parametrize("call,message", [
    (lambda: mok.sort_tokens(_i32(8), 4), r"topk_ids: shape \(8,\)"),
    (lambda: mok.sort_tokens(torch.zeros(8, 2).long(), 4), "topk_ids: dtype torch.int64"),
    (lambda: mok.sort_tokens(_i32(8, 2), 4, outs=dict(offsets=_i32(4), slots=_i32(8, 2), row_slots=_i32(16))),
     r"offsets: shape \(4,\)"),
    (lambda: mok.sort_tokens(_i32(8, 2), 4), "must be on a GPU"),
    (lambda: mok.permute(_bf(7, 64), SORT), r"x: shape \(7, 64\)"),
    (lambda: mok.permute(_bf(8, 64).half(), SORT), "x: dtype torch.float16"),
    (lambda: mok.permute(_bf(64, 8).T, SORT), "x: must be contiguous"),
    (lambda: mok.permute(_bf(8, 60), SORT), "H = 60"),
    (lambda: mok.permute(_bf(8, 72), SORT, fp8=True), "H = 72"),
    (lambda: mok.permute(_bf(8, 64), SORT, rows=False), "nothing to write"),
    (lambda: mok.permute(_bf(8, 64), dict(SORT, slots=_i32(8, 2).long())), "slots: dtype torch.int64"),
    (lambda: mok.permute(_bf(8, 64), SORT, outs=dict(rows=_bf(39, 64))), r"rows: shape \(39, 64\)"),
    (lambda: mok.permute(_bf(8, 64), SORT, fp8=True, outs=dict(rows=_bf(40, 64), elems=_u8(40, 64), scales=_f32(40, 1))),
     r"scales: shape \(40, 1\)"),
    (lambda: mok.permute(_bf(8, 64), SORT), "must be on a GPU"),
    (lambda: mok.permute_backward(_bf(8, 64), SORT), r"drows: shape \(8, 64\), expected \[40, H\]"),
    (lambda: mok.unpermute(_bf(40, 64), SORT, w=_bf(8, 2)), "w: dtype torch.bfloat16"),
    (lambda: mok.unpermute(_bf(40, 64), SORT, addend=_f32(8, 64)), "addend: dtype torch.float32"),
    (lambda: mok.unpermute(_bf(40, 64), SORT, out=_bf(8, 32)), r"out: shape \(8, 32\)"),
    (lambda: mok.unpermute_backward(_bf(8, 64), _bf(40, 64), SORT, None), "w: expected a torch.Tensor"),
    (lambda: mok.unpermute_backward(_f32(8, 64), _bf(40, 64), SORT, _f32(8, 2)), "dout: dtype torch.float32"),
    (lambda: mok.unpermute_backward(_bf(8, 64), _bf(40, 64), SORT, _f32(8, 2), grads=dict(dy=_bf(40, 64))),
     "dw: expected a torch.Tensor"),
    (lambda: mok.fp8_quantize(_bf(4, 64)), "src: expected"),
    (lambda: mok.fp8_quantize(_bf(1, 4, 40)), "K = 40"),
    (lambda: mok.fp8_quantize(_bf(1, 64, 12), True), "rows = 12"),
    (lambda: mok.fp8_quantize(_f32(1, 4, 64), glu=True), "glu takes bf16"),
    (lambda: mok.fp8_quantize(_bf(1, 4, 64), glu=True, tile=True), "no tile"),
    (lambda: mok.fp8_quantize(_bf(1, 4, 64), outs=(_u8(1, 4, 64), _f32(1, 4, 1))), r"scales: shape \(1, 4, 1\)"),
    (lambda: mok.fp8_quantize(_bf(1, 4, 64)), "must be on a GPU"),
    (lambda: mok.glu_backward(_bf(4, 12), _bf(4, 24)), "multiple of 8"),
    (lambda: mok.glu_backward(_bf(4, 16), _bf(4, 16)), r"h: shape \(4, 16\)"),
    (lambda: mok.fp8_matmul(CODES[0], TILES), r"a: expected \(elems, scales\)"),
    (lambda: mok.fp8_matmul((CODES[0], _f32(32, 2)), TILES), r"a scales: shape \(32, 2\)"),
    (lambda: mok.fp8_matmul(CODES, (_u8(64, 128), _f32(1, 2))), r"b elems: shape \(64, 128\)"),
    (lambda: mok.fp8_matmul(CODES, (_u8(64, 256), _f32(2, 64))), r"b scales: shape \(2, 64\)"),
    (lambda: mok.fp8_matmul(CODES, (_u8(60, 256), _f32(1, 2))), "N = 60"),
    (lambda: mok.fp8_matmul(CODES, TILES, _i32(3)), r"b elems: shape \(64, 256\), expected \[E, N, K\]"),
    (lambda: mok.fp8_matmul(CODES, TILES, _i32(3).long()), "offsets: dtype torch.int64"),
    (lambda: mok.fp8_matmul(CODES, TILES, out_dtype=torch.float16), "out: dtype torch.float16"),
    (lambda: mok.fp8_matmul(CODES, TILES, out=_bf(32, 32)), r"out: shape \(32, 32\)"),
    (lambda: mok.fp8_matmul(CODES, TILES), "must be on a GPU"),
    (lambda: mok.fp8_wgrad(CODES, (_u8(32, 128), _f32(1, 32))), "128 rows along the contraction"),
    (lambda: mok.fp8_wgrad(CODES, CODES, addend=_f32(32, 32)), "addend: dtype torch.float32"),
    (lambda: mok.fp8_wgrad((_u8(24, 256), _f32(2, 24)), CODES), "N = 24"),
    (lambda: mok.fp8_wgrad(CODES, CODES, _i32(4), out=_bf(2, 32, 32)), r"out: shape \(2, 32, 32\)"),
])
def test_binding_refuses(call, message):
    with pytest.raises((ValueError, TypeError), match=message):
        call()
